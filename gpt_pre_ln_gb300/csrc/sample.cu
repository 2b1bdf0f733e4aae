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
// An id is right or wrong: a sum of fp32 weights is off by 5e-7 of itself, which
// is more than many a token's share.  So where a decision lies within that bound,
// the row is done once more with weights and sums of two floats each (2^-36 of the
// row's weight at worst, 2^-38 as a rule): 1 to 5 rows of 100, at two to four times
// the time (50257 logits: 100000 cycles more).
//
// One CTA per row, which it reads once into shared memory (rows that do not fit
// are read from global memory, where they stay in L2) and goes over there: for
// the maximum; with top-p for a histogram of the weights, and a finer one around
// the border; for the weights' sums; and over the part that the random number
// falls into.  Where the kept tokens are few (top-k, or top-p of a sharp row) they
// are listed instead, and the rest is done on the list, in two floats at once.
//
// Bound by instructions and by steps that follow one another on one SM, not by
// memory: a row of 50257 takes 19 us (its maximum 3, the histogram 7, the border 4 to
// 15, the draw 4), one that is done twice 38 to 70.  64 such rows in fp32 with top-p 69
// us, 256 with top-k up to 400 34, 1024 in bf16 with mixed settings 137 (750 GB/s), 512
// rows of 8000 16.
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
__device__ __forceinline__ Two times(Two a, float b) {
  const float h = a.hi * b;
  return norm(h, fmaf(a.hi, b, -h) + a.lo * b);
}
__device__ __forceinline__ bool less(Two a, Two b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ float minus(Two a, Two b) { return (a.hi - b.hi) + (a.lo - b.lo); }
__device__ __forceinline__ Two shfl(Two a, int from) {
  return {__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}
// (loops stay loops in what follows wherever they are not the time of a pass: a
// row goes through the code once, and what it runs for the first time it waits for)
__device__ __forceinline__ Two warp_add(Two a) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    a = add(a, Two{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
  return a;
}
__device__ __forceinline__ Two warp_incl(Two a) {  // running sum over the lanes
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Two u{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
    const Two both = add(u, a);  // (by all lanes: no branch)
    a.hi = lane >= o ? both.hi : a.hi;
    a.lo = lane >= o ? both.lo : a.lo;
  }
  return a;
}

// 2^(k / 64), k = -32 .. 31, as hi + lo
__device__ const float2 kExp2[64] = {
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
    {1.398979663848877f, 8.689434061182055e-09f}
};

// The row's scale: t = (z - max) log2(e) / temperature = (z/2 - max/2) c (half
// of each, so that the difference of any two is a number).  c_lo > 0, so that a z
// of -inf gives a t of -inf.
struct Scale {
  float half_max, c_hi, c_lo;
};
// (the same roundings in both: bins are compared by it)
__device__ __forceinline__ float exponent(const Scale& s, float z) {
  const float d = __fmaf_rn(z, 0.5f, -s.half_max);
  return __fmaf_rn(d, s.c_hi, __fmul_rn(d, s.c_lo));
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 exponent2(const Scale& s, float2 z) {
  const float2 d = fma_f32x2(z, splat(0.5f), splat(-s.half_max));
  return fma_f32x2(d, splat(s.c_hi), mul_f32x2(d, splat(s.c_lo)));
}
// Bound of the error of a sum of fp32 weights 2^t, of itself: 2^-22 of the
// exponential and four roundings of sums (those of a vector's elements; sums of
// vectors are kept in two floats), and 2 * 2^-24 ln 2 |t| for the roundings of t,
// whose mean over the weights is at most log2(V / sum): that is what their entropy
// leaves.
__device__ __forceinline__ float error_of(float sum, int V) {
  return sum * (4.8e-7f + 8.4e-8f * fmaxf(log2f(static_cast<float>(V) / sum), 0.f)) + 1e-30f;
}

// Two sums or weights of two floats each, on paired instructions.
struct TwoPair {
  float2 hi, lo;
};
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma_f32x2(b, splat(-1.f), a); }
__device__ __forceinline__ TwoPair norm2(float2 a, float2 b) {  // |a| >= |b|
  const float2 s = add_f32x2(a, b);
  return {s, sub2(b, sub2(s, a))};
}
__device__ __forceinline__ TwoPair two_sum2(float2 a, float2 b) {
  const float2 s = add_f32x2(a, b), t = sub2(s, a);
  return {s, add_f32x2(sub2(a, sub2(s, t)), sub2(b, t))};
}
// (sums of a few hundred weights: their second floats stay so far below the first ones that these are put in order
// at the end, by total)
__device__ __forceinline__ TwoPair add2(TwoPair a, TwoPair b) {
  const TwoPair s = two_sum2(a.hi, b.hi);
  return {s.hi, add_f32x2(s.lo, add_f32x2(a.lo, b.lo))};
}
__device__ __forceinline__ Two total(TwoPair a) { return add(norm(a.hi.x, a.lo.x), norm(a.hi.y, a.lo.y)); }

constexpr float kLn2Hi = 0.6931471824645996f, kLn2Lo = -1.9046542121259336e-09f;  // ln 2

// The weights of two logits to about 2^-38 of themselves: 2^t = 2^n 2^(k/64) e^x with
// integers n and k, -32 <= k < 32, and |x| <= ln 2 / 128, whose series ends with x^4.
// (The parts below x are single floats: 2^-16 of the weight, and they need no more.)
// Below 2^-44 of the largest weight fp32 will do: t's roundings there are 2^-16 of the weight at most, alike for equal
// logits, but 2^21 of them are 2^-23 of the largest.  Below 2^-100 they count as 0.
__device__ __forceinline__ TwoPair weights2(const Scale& s, const float2* table, float2 z) {
  const TwoPair d = two_sum2(mul_f32x2(z, splat(0.5f)), splat(-s.half_max));
  const float2 t = mul_f32x2(d.hi, splat(s.c_hi));
  if (!(fmaxf(t.x, t.y) > -44.f)) {
    const float2 u = fma_f32x2(d.hi, splat(s.c_lo), t);
    return {make_float2(t.x > -100.f ? ex2_approx(u.x) : 0.f, t.y > -100.f ? ex2_approx(u.y) : 0.f), splat(0.f)};
  }
  const float2 t_lo =
      fma_f32x2(d.lo, splat(s.c_hi), fma_f32x2(d.hi, splat(s.c_lo), fma_f32x2(d.hi, splat(s.c_hi), make_float2(-t.x, -t.y))));
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to whole numbers
  const float2 im = fma_f32x2(t, splat(64.f), splat(kRound)), i = add_f32x2(im, splat(-kRound));
  const float2 g = fma_f32x2(i, splat(-0.015625f), t);  // exact
  const float2 x = mul_f32x2(g, splat(kLn2Hi));
  const float2 x_lo = fma_f32x2(t_lo, splat(kLn2Hi),
                                fma_f32x2(g, splat(kLn2Lo), fma_f32x2(g, splat(kLn2Hi), make_float2(-x.x, -x.y))));
  const float2 c = fma_f32x2(x, fma_f32x2(x, splat(1.f / 24.f), splat(1.f / 6.f)), splat(0.5f));
  const float2 xx = mul_f32x2(x, x);
  const float2 y = fma_f32x2(xx, c, fma_f32x2(fma_f32x2(xx, splat(0.5f), x), x_lo, x_lo));  // e^x - 1 = x + y
  const int ix = __float_as_int(im.x) - 0x4b400000 + 32, iy = __float_as_int(im.y) - 0x4b400000 + 32;  // 64 n + k + 32
  const float2 b0 = table[ix & 63], b1 = table[iy & 63];
  const float2 b = make_float2(b0.x, b1.x), b_lo = make_float2(b0.y, b1.y);
  const float2 m = mul_f32x2(b, x);
  const float2 m_lo = add_f32x2(fma_f32x2(b_lo, x, fma_f32x2(b, y, fma_f32x2(b, x, make_float2(-m.x, -m.y)))), b_lo);
  const TwoPair w = norm2(b, m), r = norm2(w.hi, add_f32x2(w.lo, m_lo));
  // (a pair may be of one such element and one that is -inf or far below)
  const bool on_x = t.x > -100.f, on_y = t.y > -100.f;
  const float2 scale = make_float2(__int_as_float(((ix >> 6) + 127) << 23), __int_as_float(((iy >> 6) + 127) << 23));
  const TwoPair out{mul_f32x2(r.hi, scale), mul_f32x2(r.lo, scale)};
  return {make_float2(on_x ? out.hi.x : 0.f, on_y ? out.hi.y : 0.f), make_float2(on_x ? out.lo.x : 0.f, on_y ? out.lo.y : 0.f)};
}
__device__ __forceinline__ Two weight2(const Scale& s, const float2* table, float z) {
  const TwoPair w = weights2(s, table, splat(z));
  return {w.hi.x, w.lo.x};
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
using Place = unsigned long long;
__device__ __forceinline__ Place place_at(uint32_t key, int id) {
  return (static_cast<Place>(key) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}
__device__ __forceinline__ Place place_of(float z, int id) { return place_at(key_of(z), id); }
__device__ __forceinline__ int id_of(Place p) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(p)); }
__device__ __forceinline__ float z_of(Place p) { return z_of(static_cast<uint32_t>(p >> 32)); }

// The last element of the order that stays.
struct Cut {
  float z;
  int id;
  __device__ __forceinline__ bool keeps(float x, int i) const { return x > z || (x == z && i <= id); }
  __device__ __forceinline__ Place place() const { return place_of(z, id); }
};
__device__ __forceinline__ Cut cut_at(Place p) { return {z_of(p), id_of(p)}; }

// 16 bytes of a row, as pairs
template <typename T>
struct Vec {
  static constexpr int kN = 16 / static_cast<int>(sizeof(T));
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&z)[kN / 2]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
      z[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
      z[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
          z[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else
          z[i] = Type16<T>::unpack2(w[i]);
    }
  }
};
template <int N>
__device__ __forceinline__ float at(const float2 (&z)[N], int i) {
  return i & 1 ? z[i >> 1].y : z[i >> 1].x;
}

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

// Shared memory: this, and behind it the row.  (Reached by name, not through
// pointers that are handed on: the compiler then knows that it is shared memory.)
struct Shared {
  union {
    uint32_t hist[kBins];
    struct {
      Two by_order[kList], by_id[kList];
    };
  };
  Place list[kList];
  Two part[32], part2[32];
  float aux[32], aux2[32];
  int num[32];
  uint32_t lo, hi;
  int count, first, last, found, bad;
  int how, bins[4];  // of draw: where top_p's border was found
  Cut cut, cut_min;
  unsigned long long passed;  // of find_bins: the last bin + 1, and the count up to it
  float margin, logprob;
  Scale scale;
  double least;
  const uint4* global;
  int V, vecs, per_warp;  // of the row, in vectors; of one warp's part
  uint64_t bar[32];
  float2 table[64];
};
constexpr size_t kFixed = (sizeof(Shared) + 15) / 16 * 16;
__device__ __forceinline__ Shared& shared() {
  extern __shared__ __align__(16) uint8_t s_raw[];
  return *reinterpret_cast<Shared*>(s_raw);
}

// A kernel's element type, threads, and whether its rows fit shared memory.
template <typename T_, int NT_, bool IN_SMEM_>
struct Kind {
  using T = T_;
  static constexpr int NT = NT_, kWarps = NT_ / 32, kN = Vec<T_>::kN;
  static constexpr bool IN_SMEM = IN_SMEM_;
};
template <typename K>
__device__ __forceinline__ const uint4* row() {
  extern __shared__ __align__(16) uint8_t s_raw[];
  if constexpr (K::IN_SMEM)
    return reinterpret_cast<const uint4*>(s_raw + kFixed);
  else
    return shared().global;
}
// Element i of the row, -inf behind its end.
template <typename K>
__device__ __forceinline__ float element(int i) {
  return i < shared().V ? to_f32<typename K::T>(reinterpret_cast<const typename K::T*>(row<K>())[i]) : -INFINITY;
}
template <typename K>
__device__ __forceinline__ void vector_of(int v, int V, float2 (&z)[K::kN / 2]) {
  Vec<typename K::T>::unpack(row<K>()[v], z);
  if ((v + 1) * K::kN > V) {
#pragma unroll
    for (int i = 0; i < K::kN / 2; ++i) {
      if (v * K::kN + 2 * i >= V) z[i].x = -INFINITY;
      if (v * K::kN + 2 * i + 1 >= V) z[i].y = -INFINITY;
    }
  }
}
// This warp's part of the row: the vectors from .. to - 1.
__device__ __forceinline__ void part_of(int warp, int& from, int& to) {
  from = min(warp * shared().per_warp, shared().vecs);
  to = min(from + shared().per_warp, shared().vecs);
}

// Adds a pair to the sums of the even elements and of the odd ones.
__device__ __forceinline__ void add_to(TwoPair& sum, float2 x) {
  const TwoPair s = two_sum2(sum.hi, x);
  sum = {s.hi, add_f32x2(sum.lo, s.lo)};
}
// Weights 2^t of a vector's elements, added up pair by pair.
template <int N>
__device__ __forceinline__ float2 sum_of(const float2 (&t)[N]) {
  float2 w[N];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = make_float2(ex2_approx(t[i].x), ex2_approx(t[i].y));
#pragma unroll
  for (int o = 1; o < N; o <<= 1)
#pragma unroll
    for (int i = 0; i < N; i += 2 * o) w[i] = add_f32x2(w[i], w[i + o]);
  return w[0];
}
template <int N>
__device__ __forceinline__ void exponents(const Scale& s, const float2 (&z)[N], float2 (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = exponent2(s, z[i]);
}
// Exponents of elements that the cut does not keep become -inf.
template <int N>
__device__ __forceinline__ void cut_off(const Cut& cut, const float2 (&z)[N], int id, float2 (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!cut.keeps(z[i].x, id + 2 * i)) t[i].x = -INFINITY;
    if (!cut.keeps(z[i].y, id + 2 * i + 1)) t[i].y = -INFINITY;
  }
}
__device__ __forceinline__ void add_to(Two& sum, float x) {
  float s, e;
  two_sum(sum.hi, x, s, e);
  sum = {s, sum.lo + e};
}
// Elements i and i + 1 (i even), -inf behind the row's end.
template <typename K>
__device__ __forceinline__ float2 elements(int i, int V) {
  float2 z;
  if constexpr (sizeof(typename K::T) == 4)
    z = reinterpret_cast<const float2*>(row<K>())[i >> 1];
  else
    z = Type16<typename K::T>::unpack2(reinterpret_cast<const uint32_t*>(row<K>())[i >> 1]);
  return make_float2(i < V ? z.x : -INFINITY, i + 1 < V ? z.y : -INFINITY);
}
// Weight of the elements of vectors from .. to - 1 that the cut keeps, a warp's
// lanes side by side: a lane's.
template <typename K, bool TWO>
__device__ __forceinline__ Two lane_sum(const Scale& s, int V, const Cut& cut, int from, int to) {
  const int lane = threadIdx.x & 31;
  TwoPair sum{splat(0.f), splat(0.f)};
  if constexpr (TWO) {
#pragma unroll 1
    for (int i = from * K::kN + 2 * lane; i < to * K::kN; i += 64) {
      float2 z = elements<K>(i, V);
      if (!cut.keeps(z.x, i)) z.x = -INFINITY;
      if (!cut.keeps(z.y, i + 1)) z.y = -INFINITY;
      sum = add2(sum, weights2(s, shared().table, z));
    }
  } else {
    const bool whole = cut.z == -INFINITY;  // (what is -inf weighs nothing)
#pragma unroll 2
    for (int v = from + lane; v < to; v += 32) {
      float2 z[K::kN / 2], t[K::kN / 2];
      vector_of<K>(v, V, z);
      exponents(s, z, t);
      if (!whole) cut_off(cut, z, v * K::kN, t);
      add_to(sum, sum_of(t));
    }
  }
  return total(sum);
}
// The weight of vector v's elements that the cut keeps.
template <typename K, bool TWO>
__device__ __forceinline__ Two vector_sum(const Scale& s, int V, const Cut& cut, int v) {
  TwoPair sum{splat(0.f), splat(0.f)};
  if constexpr (TWO) {
#pragma unroll 1
    for (int i = v * K::kN; i < (v + 1) * K::kN; i += 2) {
      float2 z = elements<K>(i, V);
      if (!cut.keeps(z.x, i)) z.x = -INFINITY;
      if (!cut.keeps(z.y, i + 1)) z.y = -INFINITY;
      sum = add2(sum, weights2(s, shared().table, z));
    }
  } else {
    float2 z[K::kN / 2], t[K::kN / 2];
    vector_of<K>(v, V, z);
    exponents(s, z, t);
    cut_off(cut, z, v * K::kN, t);
    add_to(sum, sum_of(t));
  }
  return total(sum);
}
// lane_sum over the lanes.
template <typename K, bool TWO>
__device__ __noinline__ Two sum_vectors(Cut cut, int from, int to) {
  const Two sum = lane_sum<K, TWO>(shared().scale, shared().V, cut, from, to);
  __syncwarp();
  return warp_add(sum);
}

// Sum over the block; every thread gets it.
template <typename K>
__device__ __noinline__ Two block_add(Two a) {
  Shared& sh = shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = warp_add(norm(a.hi, a.lo));
  if (lane == 0) sh.part[warp] = a;
  __syncthreads();
  a = lane < K::kWarps ? sh.part[lane] : Two{0.f, 0.f};
  a = warp_add(a);
  __syncthreads();
  return a;
}
template <typename K>
__device__ __forceinline__ int block_add(int a) {
  Shared& sh = shared();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = __reduce_add_sync(0xffffffffu, a);
  if (lane == 0) sh.num[warp] = a;
  __syncthreads();
  a = __reduce_add_sync(0xffffffffu, lane < K::kWarps ? sh.num[lane] : 0);
  __syncthreads();
  return a;
}

// ------------------------------------------------------------ histogram
// Bins of equal width in z, 64 to a factor of two of the weight, bin b around
// 2^(-b / 64); the last one takes all below 2^-32.
constexpr float kMagic = 8388608.f;  // 2^23: adding it rounds to whole numbers
__device__ __forceinline__ float bin_edge(int b) { return kMagic + static_cast<float>(b); }
__device__ __forceinline__ float bin_at(float t) { return __fmaf_rn(t, -64.f, kMagic); }  // compared with an edge
// Counts a pair of weights, those above 2^-32, in units of their bins' steps
// (2^(-b / 64) is `one` of them): integers, so that sums do not depend on the order
// of the additions.  e^x with |x| <= ln 2 / 128 is taken as 1 + x: 1.5e-5 off at
// most.  Both steps round to whole numbers, and equal logits do so alike: a sum of
// bins may be off by 1 / one of itself.
__device__ __forceinline__ void count_weights(uint32_t* hist, float2 t, float one) {
  const float unit = 0.010830424696249145f * one;  // ln 2 / 64
  const float2 m = fma_f32x2(t, splat(-64.f), splat(kMagic)), b = add_f32x2(m, splat(-kMagic));
  const float2 n = fma_f32x2(t, splat(64.f * unit), fma_f32x2(b, splat(unit), splat(one + kMagic)));
  if (t.x > -31.9f) atomicAdd(hist + (__float_as_int(m.x) - 0x4b000000), __float_as_uint(n.x) - 0x4b000000u);
  if (t.y > -31.9f) atomicAdd(hist + (__float_as_int(m.y) - 0x4b000000), __float_as_uint(n.y) - 0x4b000000u);
}
// The error of a sum of bins, of itself: the above (a weight is 2^(-1 / 128) of its bin's at least) and fp32 sums.
__device__ __forceinline__ float error_of_bins(float one) { return 2e-5f + 1.01f / one; }

// Where the running sum over the bins, each h / one times 2^(-b / 64) (or 1, if
// flat), comes within `margin` of `want`, and where it passes it by as much: bins
// first and last (the last bin of all where that is not found); in `count` the sum
// of h / one of the bins up to last.
template <typename K>
__device__ __noinline__ void find_bins(bool flat, float one, float want, float margin, int& first, int& last,
                                       float& count) {
  constexpr int kPer = kBins / K::NT;
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float scale = 1.f / one, slope = flat ? 0.f : -0.015625f;
  float run = 0.f, n = 0.f;
#pragma unroll 2
  for (int i = 0; i < kPer; ++i) {
    const float h = static_cast<float>(sh.hist[tid * kPer + i]) * scale;
    n += h;
    run = fmaf(h, ex2_approx(static_cast<float>(tid * kPer + i) * slope), run);
  }
  const float mine = run, mine_n = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, run, o), un = __shfl_up_sync(0xffffffffu, n, o);
    if (lane >= o) run += u, n += un;
  }
  if (lane == 31) {
    sh.aux[warp] = run;
    sh.aux2[warp] = n;
  }
  if (tid == 0) {
    sh.first = kBins;
    sh.passed = 0;
  }
  __syncthreads();
  float ahead = lane < warp ? sh.aux[lane] : 0.f, ahead_n = lane < warp ? sh.aux2[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    ahead_n += __shfl_xor_sync(0xffffffffu, ahead_n, o);
  }
  run += ahead - mine;
  n += ahead_n - mine_n;
#pragma unroll 2
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    const float h = static_cast<float>(sh.hist[b]) * scale, before = run;
    n += h;
    run = fmaf(h, ex2_approx(static_cast<float>(b) * slope), run);
    if ((b == 0 || before < want - margin) && run >= want - margin) atomicMin(&sh.first, b);
    if ((b == 0 || before < want + margin) && run >= want + margin)
      atomicMax(&sh.passed, (static_cast<unsigned long long>(b + 1) << 32) | __float_as_uint(n));
  }
  __syncthreads();
  // (where one thread's sum ends a rounding below the next one's start a border may be found by neither, where it
  // ends above by both: then the later one's bin and count, whoever comes first)
  const int bin = static_cast<int>(sh.passed >> 32) - 1;
  first = sh.first;
  last = first < kBins && bin >= first ? bin : kBins - 1;
  count = bin >= 0 ? __uint_as_float(static_cast<uint32_t>(sh.passed)) : 1e9f;
  __syncthreads();
}

// Sums up to each of the kList values at a (in place, its own included), over the
// block.
template <typename K, bool BY_ID>
__device__ __noinline__ void scan_list() {
  constexpr int kPer = K::NT >= kList ? 1 : kList / K::NT;
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool on = tid * kPer < kList;
  Two x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    x[i] = on ? (BY_ID ? sh.by_id : sh.by_order)[tid * kPer + i] : Two{0.f, 0.f};
    if (i > 0) x[i] = add(x[i - 1], x[i]);
  }
  Two incl = warp_incl(x[kPer - 1]);
  if (lane == 31) sh.part[warp] = incl;
  __syncthreads();
  const Two parts = warp_incl(lane < K::kWarps ? sh.part[lane] : Two{0.f, 0.f});
  Two before = shfl(incl, (lane + 31) & 31);
  if (lane == 0) before = {0.f, 0.f};
  const Two ahead = shfl(parts, (warp + 31) & 31);
  if (warp > 0) before = add(ahead, before);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (on) (BY_ID ? sh.by_id : sh.by_order)[tid * kPer + i] = add(before, x[i]);
  __syncthreads();
}

// An element of the list and its ranks: in the order, and among the ids.
struct Listed {
  Place p;
  Two w;
  int rank, rank_id;
};
template <typename K>
constexpr int kListed = K::NT >= kList ? 1 : kList / K::NT;  // per thread

// The n elements of the list: ranks and weights, and by_order the sums of the
// weights in the order.  (Each against all: 3000 cycles for 100 of them, 15000 for
// 500.)
template <typename K>
__device__ __forceinline__ void rank_list(int n, Listed (&mine)[kListed<K>]) {
  Shared& sh = shared();
  for (int i = threadIdx.x; i < kList; i += K::NT) {
    sh.by_order[i] = {0.f, 0.f};
    if (i >= n) sh.list[i] = 0;  // ranks behind all others
  }
  __syncthreads();
  const Scale s = sh.scale;
  const ulonglong2* list = reinterpret_cast<const ulonglong2*>(sh.list);
#pragma unroll 1
  for (int e = 0; e < kListed<K>; ++e) {
    const int i = threadIdx.x + e * K::NT;
    Listed x{0, {0.f, 0.f}, 0, 0};
    if (i < n) {
      x.p = sh.list[i];
      const uint32_t low = static_cast<uint32_t>(x.p);
#pragma unroll 4
      for (int k = 0; k < (n + 1) / 2; ++k) {
        const ulonglong2 q = list[k];
        x.rank += (q.x > x.p) + (q.y > x.p);
        // (a lower id has the larger number)
        x.rank_id += (static_cast<uint32_t>(q.x) > low) + (static_cast<uint32_t>(q.y) > low);
      }
      x.w = weight2(s, sh.table, z_of(x.p));
      sh.by_order[x.rank] = x.w;
    }
    mine[e] = x;
  }
  __syncthreads();
  scan_list<K, false>();
}

// Of the list's elements, those that stay: the first `most`, kept by cut_min, and
// before which, with `ahead` before the list, less than `target` stands; one at
// least if `one`.  Their number; `loose`: the weight of those that an error of `err`
// in the difference leaves undecided.
template <typename K>
__device__ __forceinline__ int keep_listed(int n, const Listed (&mine)[kListed<K>], int most, const Cut& cut_min,
                                           Two ahead, Two target, float err, bool one, float& loose) {
  Shared& sh = shared();
  int in = 0;
  Two unsure{0.f, 0.f};
#pragma unroll 1
  for (int e = 0; e < kListed<K>; ++e) {
    if (threadIdx.x + e * K::NT >= n) break;
    const Listed& x = mine[e];
    Two before = ahead;
    if (x.rank > 0) before = add(ahead, sh.by_order[x.rank - 1]);
    if (x.rank < most && cut_min.keeps(z_of(x.p), id_of(x.p))) {
      in += less(before, target) || (one && x.rank == 0);
      if (err > 0.f && fabsf(minus(before, target)) <= err) add_to(unsure, x.w.hi);
    } else if (one && x.rank == 0) {
      ++in;
    }
  }
  __syncwarp();
  const int kept = block_add<K>(in);
  loose = err > 0.f ? block_add<K>(unsure).hi : 0.f;
  return kept;
}
__device__ __forceinline__ Two listed_sum(int kept, Two ahead) {
  return kept > 0 ? add(ahead, shared().by_order[kept - 1]) : ahead;
}

// ------------------------------------------------------------ crowded borders
// The last of the elements kept by `cut` that stays: the `count` first of them
// (MASS false), or those before which less than `target` of weight stands (MASS).
// For any row, at its own pace: histograms over ever smaller intervals of the
// order, until few enough elements are left to rank; the first one of bins of equal
// width in z, later ones, where equal or nearly equal logits crowd a bin, of bins of
// equal width in the place.  The first one's bins go from the maximum to the least
// that is not -inf; with MASS no further than a weight of 2^-100, behind which no
// border lies (what is there weighs 2^-79 in all).  A bin counts its weights in steps
// of the heaviest that fits it, so it must not span more than a fraction of a factor
// of two, however low the row's least logit (a mask's -1e9) is.  In *loose the weight
// of the elements that sums off by `err` leave undecided (INFINITY: none decided).
template <typename K, bool MASS, bool TWO>
__device__ __noinline__ Cut select(Cut cut, int count, Two target, float err, float* loose) {
  constexpr int kPer = kBins / K::NT;
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = sh.V;
  const Scale s = sh.scale;
  int from, to;
  part_of(warp, from, to);
  from *= K::kN;
  to = min(to * K::kN, V);
  Place lo = cut.place(), hi = place_of(2.f * s.half_max, 0);  // the interval
  if (MASS) lo = max(lo, static_cast<Place>(key_of(2.f * (s.half_max - 100.f / s.c_hi))) << 32);
  int n = V;         // elements that it holds, at most
  int before_n = 0;  // elements ahead of it
  auto weight = [&](float z, Two& sum) {
    if constexpr (TWO)
      sum = add(sum, weight2(s, sh.table, z));
    else
      add_to(sum, ex2_approx(exponent(s, z)));
  };
  // the least that is not -inf, and with it the first histogram's bins
  if (tid == 0) sh.lo = 0xffffffffu;
  __syncthreads();
  uint32_t least = 0xffffffffu;
  int there = 0;  // (what is -inf is never drawn: it might as well not be there)
#pragma unroll 1
  for (int i = from + lane; i < to; i += 32) {
    const float z = element<K>(i);
    if (z > -INFINITY && place_of(z, i) >= lo) {
      least = min(least, key_of(z));
      ++there;
    }
  }
  __syncwarp();
  least = __reduce_min_sync(0xffffffffu, least);
  if (lane == 0) atomicMin(&sh.lo, least);
  there = block_add<K>(there);
  if (!MASS && there <= count) return cut;
  const float per_z = static_cast<float>(kBins - 8) / (s.half_max - 0.5f * z_of(sh.lo));  // (halves: no overflow)
  lo = max(lo, static_cast<Place>(sh.lo) << 32);
  __syncthreads();
  auto bin_of = [&](float z) {
    return static_cast<int>(fminf((s.half_max - 0.5f * z) * per_z, static_cast<float>(kBins - 1)));
  };
  bool linear = per_z < 3e38f;
#pragma unroll 1
  while (true) {
    if (lo >> 32 == hi >> 32) {  // one value: of its places the ids there are
      lo = max(lo, place_at(static_cast<uint32_t>(lo >> 32), V - 1));
      hi = min(hi, place_at(static_cast<uint32_t>(hi >> 32), 0));
    }
    const int shift = max(0, 64 - __clzll(static_cast<long long>(hi - lo)) - 11);
    const int digits = 31 - min(31, 32 - __clz(n));  // n elements of at most 2^digits
    const float one = static_cast<float>(1u << digits);
    const float top = linear ? 0.f : exponent(s, z_of(hi));  // the heaviest weight in it
    const float fall = linear ? s.c_hi / per_z : 0.f;  // of the heaviest weight's exponent, per bin
    for (int i = tid; i < kBins; i += K::NT) sh.hist[i] = 0;
    __syncthreads();
    Two ahead{0.f, 0.f};  // weight ahead of it
#pragma unroll 1
    for (int i = from + lane; i < to; i += 32) {
      const float z = element<K>(i);
      const Place p = place_of(z, i);
      if (p < lo || z == -INFINITY) continue;
      const float t = exponent(s, z);
      if (p > hi) {
        if (MASS) add_to(ahead, ex2_approx(t));
        continue;
      }
      const int b = linear ? bin_of(z) : kBins - 1 - static_cast<int>((p - lo) >> shift);
      const float over = t - top + static_cast<float>(b) * fall;
      atomicAdd(&sh.hist[b], MASS ? __float2uint_rn(fminf(ex2_approx(over), 1.02f) * 0.98f * one) : 1u);
    }
    __syncwarp();
    ahead = block_add<K>(ahead);
    // the bins that the border may be in (weights carry 0.98 of themselves, so that a bin's sum fits)
    auto of_bin = [&](int b) {
      const float h = static_cast<float>(sh.hist[b]);
      return MASS ? h / (0.98f * one) * ex2_approx(top - static_cast<float>(b) * fall) : h;
    };
    float run = 0.f;
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) run += of_bin(tid * kPer + i);
    const float mine = run;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const float u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) sh.aux[warp] = run;
    if (tid == 0) {
      sh.first = sh.last = kBins - 1;
      sh.count = 0;
      sh.lo = 0xffffffffu;
      sh.hi = 0;
    }
    __syncthreads();
    float all = ahead.hi;
#pragma unroll 1
    for (int w = 0; w < K::kWarps; ++w) {
      if (w < warp) run += sh.aux[w];
      all += sh.aux[w];
    }
    run += (MASS ? ahead.hi : static_cast<float>(before_n)) - mine;
    // a step of the histogram per element, and the roundings of the sums (counts are exact)
    const float margin =
        MASS ? (linear ? 1.1f * all : static_cast<float>(n) * ex2_approx(top)) / one + 1e-4f * all + err : 0.f;
    const float want = MASS ? target.hi : static_cast<float>(count);
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      run += of_bin(tid * kPer + i);
      if (run >= want - margin) atomicMin(&sh.first, tid * kPer + i);
      if (run >= want + margin) {
        atomicMin(&sh.last, tid * kPer + i);
        break;
      }
    }
    __syncthreads();
    // the elements in them, and the weight ahead of them
    const int first = sh.first, last = sh.last;
    const Place was = hi - lo, off = (static_cast<Place>(kBins - 1 - first) << shift) + ((1ull << shift) - 1);
    const Place in_lo = lo + (static_cast<Place>(kBins - 1 - last) << shift), in_hi = off >= was ? hi : lo + off;
    Two above{0.f, 0.f};
    uint32_t k_lo = 0xffffffffu, k_hi = 0;
    int ahead_n = 0;
#pragma unroll 1
    for (int i = from + lane; i < to; i += 32) {
      const float z = element<K>(i);
      const Place p = place_of(z, i);
      if (p < lo || z == -INFINITY) continue;
      int where;  // 1 ahead, 0 in them, -1 behind
      if (linear) {
        const int b = bin_of(z);
        where = b < first ? 1 : b > last ? -1 : 0;
      } else {
        where = p > in_hi ? 1 : p < in_lo ? -1 : 0;
      }
      if (where > 0) {
        ++ahead_n;
        if (MASS) weight(z, above);
      } else if (where == 0) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < kList) sh.list[at] = p;
        k_lo = min(k_lo, static_cast<uint32_t>(p >> 32));
        k_hi = max(k_hi, static_cast<uint32_t>(p >> 32));
      }
    }
    __syncwarp();
    k_lo = __reduce_min_sync(0xffffffffu, k_lo);
    k_hi = __reduce_max_sync(0xffffffffu, k_hi);
    if (lane == 0) {
      atomicMin(&sh.lo, k_lo);
      atomicMax(&sh.hi, k_hi);
    }
    above = block_add<K>(above);
    ahead_n = block_add<K>(ahead_n);
    n = sh.count;
    if (n > kList) {
      if (linear) {
        lo = max(lo, static_cast<Place>(sh.lo) << 32);
        hi = min(hi, (static_cast<Place>(sh.hi) << 32) | 0xffffffffu);
      } else {
        lo = in_lo;
        hi = in_hi;
      }
      before_n = ahead_n;
      if (MASS && !linear && hi - lo > was / 2) {
        // weights of very different sizes, too fine for the histogram's step: by halves
        const Place mid = lo + (hi - lo) / 2;
        Two sum{0.f, 0.f};
        int more_n = 0;
#pragma unroll 1
        for (int i = from + lane; i < to; i += 32) {
          const float z = element<K>(i);
          const Place p = place_of(z, i);
          if (p < mid) continue;
          more_n += p <= hi;
          weight(z, sum);
        }
        __syncwarp();
        sum = block_add<K>(sum);
        more_n = block_add<K>(more_n);
        if (!TWO && fabsf(minus(sum, target)) <= err) {  // left to the sums of two floats
          *loose = INFINITY;
          return cut;
        }
        if (!less(sum, target)) {
          lo = mid;
          n = more_n;
        } else {
          hi = mid - 1;
          n -= more_n;
          before_n += more_n;
        }
      }
      linear = false;
      __syncthreads();
      continue;
    }
    Listed mine_l[kListed<K>];
    rank_list<K>(n, mine_l);
    int kept;
    if (MASS) {
      float unsure;
      kept = keep_listed<K>(n, mine_l, n, Cut{-INFINITY, V}, above, target, err, true, unsure);
      *loose = unsure;
    } else {
      kept = min(count - ahead_n, n);
    }
#pragma unroll 1
    for (int e = 0; e < kListed<K>; ++e)
      if (tid + e * K::NT < n && mine_l[e].rank == kept - 1) sh.cut = cut_at(mine_l[e].p);
    __syncthreads();
    const Cut c = sh.cut;
    __syncthreads();
    return c;
  }
}

// ------------------------------------------------------------ drawing
// The first lane whose end passes the target, or the last that has weight where
// rounding leaves none.
__device__ __forceinline__ int first_past(Two end, Two target, bool has) {
  const unsigned past = __ballot_sync(0xffffffffu, has && less(target, end));
  if (past) return __ffs(static_cast<int>(past)) - 1;
  const unsigned any = __ballot_sync(0xffffffffu, has);
  return any ? 31 - __clz(static_cast<int>(any)) : 0;
}

// (t of 100 has steps of 2^-17: in two floats up to the last rounding)
__device__ __forceinline__ float logprob_of(const Scale& s, float z, Two all) {
  float d, d_lo, r, r_lo;
  two_sum(0.5f * z, -s.half_max, d, d_lo);
  const float t = d * s.c_hi, t_lo = fmaf(d, s.c_hi, -t) + fmaf(d, s.c_lo, d_lo * s.c_hi);
  const float p = t * kLn2Hi, p_lo = fmaf(t, kLn2Hi, -p) + fmaf(t, kLn2Lo, t_lo * kLn2Hi);
  // (the largest weighs 1, so that neither part is above 0; of a share near 1 the sum's second float matters)
  two_sum(p, -log1pf((all.hi - 1.f) + all.lo), r, r_lo);
  return r + (r_lo + p_lo);
}
// Whether a log probability stays within 1e-5 where `all` may be off by err: less what its own rounding (2^-24 of
// it) and the logarithm of a sum of up to 2^21 (a step of 2^-20, and the rounding of its argument) take of that.
__device__ __forceinline__ bool near_enough(float err, Two all, float logprob) {
  return err <= (8.9e-6f + 6e-8f * logprob) * all.hi;
}

// Draws from the `kept` first of the ranked list, whose weight is `all`, `loose`
// of which may not belong.  The sums by id are those of a parallel scan, whose second
// floats may differ by their roundings where nothing is added, or fall: so the row
// belongs to the lowest kept id whose sum passes the target, and to no other.
template <typename K>
__device__ __forceinline__ bool draw_listed(int n, const Listed (&mine)[kListed<K>], int kept, Two all, float loose,
                                            float u, int& token, float& logprob) {
  Shared& sh = shared();
  const Two target = times(all, u);
  for (int i = threadIdx.x; i < kList; i += K::NT) sh.by_id[i] = {0.f, 0.f};
  if (threadIdx.x == 0) {
    sh.first = kList;
    sh.last = -1;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < kListed<K>; ++e)
    if (threadIdx.x + e * K::NT < n && mine[e].rank < kept) sh.by_id[mine[e].rank_id] = mine[e].w;
  __syncthreads();
  scan_list<K, true>();
#pragma unroll 1
  for (int e = 0; e < kListed<K>; ++e) {
    if (threadIdx.x + e * K::NT >= n) break;
    const Listed& x = mine[e];
    if (x.rank >= kept || !(x.w.hi > 0.f)) continue;
    if (less(target, sh.by_id[x.rank_id])) atomicMin(&sh.first, x.rank_id);
    atomicMax(&sh.last, x.rank_id);
  }
  __syncthreads();
  // (rounding may leave the last one's end below the target)
  const int owner = min(sh.first, sh.last);
#pragma unroll 1
  for (int e = 0; e < kListed<K>; ++e) {
    if (threadIdx.x + e * K::NT >= n) break;
    const Listed& x = mine[e];
    if (x.rank_id != owner) continue;
    Two before{0.f, 0.f};
    if (owner > 0) before = sh.by_id[owner - 1];
    sh.found = id_of(x.p);
    // how far the random number is from the ends of this token's share (nothing is before the first)
    sh.margin = minus(sh.by_id[owner], target);
    if (before.hi > 0.f || loose > 0.f) sh.margin = fminf(sh.margin, minus(target, before));
    sh.logprob = logprob_of(sh.scale, z_of(x.p), all);
  }
  __syncthreads();
  token = sh.found;
  logprob = sh.logprob;
  const float margin = sh.margin;
  __syncthreads();
  return loose == 0.f || (margin > 2.f * loose && near_enough(loose, all, logprob));
}

// The elements with z >= least that the cut keeps into the list; how many there
// are.
template <typename K>
__device__ __noinline__ int list_from(Cut cut, float least) {
  Shared& sh = shared();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  const int V = sh.V;
  int from, to;
  part_of(threadIdx.x >> 5, from, to);
#pragma unroll 1
  for (int v = from + (threadIdx.x & 31); v < to; v += 32) {
    float2 z[K::kN / 2];
    vector_of<K>(v, V, z);
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < K::kN; ++i) in |= at(z, i) >= least ? 1u << i : 0u;
    for (; in; in &= in - 1) {
      const int id = v * K::kN + __ffs(static_cast<int>(in)) - 1;
      const float x = element<K>(id);
      if (id >= V || !cut.keeps(x, id)) continue;
      const int at = atomicAdd(&sh.count, 1);
      if (at < kList) sh.list[at] = place_of(x, id);
    }
  }
  __syncthreads();
  return sh.count;
}
// The least z whose bin is at most b (of those the row has, or a step beside it:
// bins fall as z grows).
__device__ __forceinline__ float least_in_bin(const Scale& s, int b) {
  // t = -(b + 1/2) / 64, and outward by more than its roundings
  const float t = -(static_cast<float>(b) + 0.5f) * 0.015625f;
  const float d = t / s.c_hi;
  return 2.f * (s.half_max + d) - (fabsf(s.half_max) + fabsf(d)) * 1e-6f;
}

// The histogram of the weights of the elements kept by `cut`, and their sum.
template <typename K>
__device__ __forceinline__ Two weigh(Cut cut, float one) {
  Shared& sh = shared();
  for (int i = threadIdx.x; i < kBins; i += K::NT) sh.hist[i] = 0;
  __syncthreads();
  const Scale s = sh.scale;
  const int V = sh.V;
  int from, to;
  part_of(threadIdx.x >> 5, from, to);
  TwoPair sum{splat(0.f), splat(0.f)};
  const bool whole = cut.z == -INFINITY;
#pragma unroll 1
  for (int v = from + (threadIdx.x & 31); v < to; v += 32) {
    float2 z[K::kN / 2], t[K::kN / 2];
    vector_of<K>(v, V, z);
    exponents(s, z, t);
    if (!whole) cut_off(cut, z, v * K::kN, t);
    add_to(sum, sum_of(t));
#pragma unroll
    for (int i = 0; i < K::kN / 2; ++i) count_weights(sh.hist, t[i], one);
  }
  __syncwarp();
  return block_add<K>(total(sum));
}

// What a sub-bin is of: bins first .. last, cut into kBins.
struct SubBins {
  float edge_first, edge_last, top, per_t, middle;
  __device__ __forceinline__ SubBins(int first, int last)
      : edge_first(bin_edge(first)), edge_last(bin_edge(last)), top((static_cast<float>(first) - 0.5f) * 0.015625f),
        per_t(64.f * static_cast<float>(kBins) / static_cast<float>(last - first + 1)),
        middle(static_cast<float>(first + last) * 0.0078125f) {}
  __device__ __forceinline__ float place(float t) const { return (-t - top) * per_t; }
  __device__ __forceinline__ int of(float t) const { return max(0, min(kBins - 1, static_cast<int>(place(t)))); }
};

// This warp's part of the row: the weight of the elements kept by `cut` ahead of
// bin `first`; those in bins first .. last are counted in sub-bins, in units of the
// weight of their middle / one.
template <typename K>
__device__ __noinline__ Two sum_ahead(Cut cut, int first, int last, float one) {
  Shared& sh = shared();
  const Scale s = sh.scale;
  const int V = sh.V;
  const SubBins sub(first, last);
  const bool whole = cut.z == -INFINITY;
  int from, to;
  part_of(threadIdx.x >> 5, from, to);
  TwoPair sum{splat(0.f), splat(0.f)};
#pragma unroll 1
  for (int v = from + (threadIdx.x & 31); v < to; v += 32) {
    float2 z[K::kN / 2], t[K::kN / 2];
    vector_of<K>(v, V, z);
    exponents(s, z, t);
    if (!whole) cut_off(cut, z, v * K::kN, t);
    uint32_t in = 0, more = 0;
#pragma unroll
    for (int i = 0; i < K::kN; ++i) {
      const float b = bin_at(at(t, i));
      if (b <= sub.edge_last) {
        if (b >= sub.edge_first)
          in |= 1u << i;
        else
          more |= 1u << i;
      }
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < K::kN / 2; ++i) {
        if (!((more >> (2 * i)) & 1)) t[i].x = -INFINITY;
        if (!((more >> (2 * i + 1)) & 1)) t[i].y = -INFINITY;
      }
      add_to(sum, sum_of(t));
    }
    for (; in; in &= in - 1) {
      const float x = exponent(s, element<K>(v * K::kN + __ffs(static_cast<int>(in)) - 1));
      atomicAdd(&sh.hist[sub.of(x)], __float2uint_rn(ex2_approx(x + sub.middle) * one));
    }
  }
  __syncwarp();
  return warp_add(total(sum));
}
// And of those in bins first .. last the weight of the ones ahead of sub-bin
// sub_first, and the ones up to sub_last into the list.
template <typename K>
__device__ __noinline__ Two list_border(Cut cut, int first, int last, int sub_first, int sub_last) {
  Shared& sh = shared();
  const Scale s = sh.scale;
  const int V = sh.V;
  const SubBins sub(first, last);
  int from, to;
  part_of(threadIdx.x >> 5, from, to);
  Two sum{0.f, 0.f};
#pragma unroll 1
  for (int v = from + (threadIdx.x & 31); v < to; v += 32) {
    float2 z[K::kN / 2], t[K::kN / 2];
    vector_of<K>(v, V, z);
    exponents(s, z, t);
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < K::kN; ++i) {
      const float b = bin_at(at(t, i));
      in |= b >= sub.edge_first && b <= sub.edge_last ? 1u << i : 0u;
    }
    for (; in; in &= in - 1) {
      const int id = v * K::kN + __ffs(static_cast<int>(in)) - 1;
      const float x = element<K>(id), tx = exponent(s, x);
      if (!cut.keeps(x, id)) continue;
      const int b = sub.of(tx);
      if (b < sub_first) {
        add_to(sum, ex2_approx(tx));
      } else if (b <= sub_last) {
        const int place = atomicAdd(&sh.count, 1);
        if (place < kList) sh.list[place] = place_of(x, id);
      }
    }
  }
  __syncwarp();
  return warp_add(norm(sum.hi, sum.lo));
}
// The sums of both in two floats each, and in `rest` the weight of the others.
template <typename K>
__device__ __noinline__ Two sum_both(Cut cut, int first, int last, int sub_first, Two& rest) {
  const Scale s = shared().scale;
  const int V = shared().V;
  const SubBins sub(first, last);
  int from, to;
  part_of(threadIdx.x >> 5, from, to);
  const float end_ahead = sub_first > 0 ? static_cast<float>(sub_first) : -INFINITY;
  TwoPair ahead{splat(0.f), splat(0.f)}, others = ahead;
#pragma unroll 1
  for (int i = from * K::kN + 2 * (threadIdx.x & 31); i < to * K::kN; i += 64) {
    float2 z = elements<K>(i, V);
    if (!cut.keeps(z.x, i)) z.x = -INFINITY;
    if (!cut.keeps(z.y, i + 1)) z.y = -INFINITY;
    const TwoPair w = weights2(s, shared().table, z);
    const float2 t = exponent2(s, z);
    auto is_ahead = [&](float t) {  // (of(t) < sub_first, without the conversion)
      const float b = bin_at(t);
      return (b < sub.edge_first) | ((b <= sub.edge_last) & (sub.place(t) < end_ahead));
    };
    const bool x = is_ahead(t.x), y = is_ahead(t.y);
    ahead = add2(ahead, {make_float2(x ? w.hi.x : 0.f, y ? w.hi.y : 0.f), make_float2(x ? w.lo.x : 0.f, y ? w.lo.y : 0.f)});
    others = add2(others, {make_float2(x ? 0.f : w.hi.x, y ? 0.f : w.hi.y), make_float2(x ? 0.f : w.lo.x, y ? 0.f : w.lo.y)});
  }
  __syncwarp();
  rest = warp_add(total(others));
  return warp_add(total(ahead));
}

// How the elements that top_p keeps are found.
enum { kFew, kMany, kCrowded };

// Draws the row's token from the elements kept by `cut`, of those the first that
// top_p leaves, and kept by cut_min.  False where fp32 sums do not decide it.
template <typename K, bool TWO>
__device__ __noinline__ bool draw(Cut cut, float top_p, float u, int& token, float& logprob) {
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = sh.V;
  const Cut cut_min = sh.cut_min;
  float loose = 0.f;
  bool summed = false;  // sh.part2 has the sums of the warps' parts
  if (top_p < 1.f) {
    // where the border is: found in fp32, with the margin that its sums need
    int first, last, sub_first = 0, sub_last = kBins - 1;
    Two all, part{0.f, 0.f}, target;
    float err = 0.f;
    if constexpr (!TWO) {
      const int digits = 31 - (32 - __clz(V));  // as many elements of 1.01 * 2^digits fit 32 bits
      const float one = static_cast<float>(1u << min(digits, 15));
      all = weigh<K>(cut, one);
      err = 2.f * error_of(all.hi, V);  // of a border's two sides
      target = times(all, top_p);
      float count;
      find_bins<K>(false, one, target.hi, error_of_bins(one) * all.hi + err, first, last, count);
      // (the border is far below the maximum, or among very different weights)
      int how = last >= kBins - 64 || last - first > 64 ? kCrowded : count * 1.02f <= kList / 2 ? kFew : kMany;
      if (how == kMany) {
        // the sums of the elements ahead of the border's bins, by parts; a finer histogram of those bins; then
        // the sums with its bins ahead of the border, and the elements around it
        for (int i = tid; i < kBins; i += K::NT) sh.hist[i] = 0;
        if (tid == 0) sh.count = 0;
        __syncthreads();
        part = sum_ahead<K>(cut, first, last, one);
        if (lane == 0) sh.part2[warp] = part;
        __syncthreads();
        const Two ahead = warp_add(lane < K::kWarps ? sh.part2[lane] : Two{0.f, 0.f});
        const float unit = ex2_approx(static_cast<float>(first + last) * -0.0078125f);
        // (the sum ahead is off by err, the histogram by its step and its sums' roundings)
        const float margin = err + (1.f / one + 2e-6f) * all.hi;
        find_bins<K>(true, one / unit, minus(target, ahead), margin, sub_first, sub_last, count);
        if (sub_first >= kBins) sub_first = 0, sub_last = kBins - 1;
      }
      if (tid == 0) {
        sh.how = how;
        sh.bins[0] = first, sh.bins[1] = last, sh.bins[2] = sub_first, sh.bins[3] = sub_last;
      }
    } else {
      first = sh.bins[0], last = sh.bins[1], sub_first = sh.bins[2], sub_last = sh.bins[3];
      if (sh.how == kMany) {
        Two rest;
        part = sum_both<K>(cut, first, last, sub_first, rest);
        all = block_add<K>(lane == 0 ? add(part, rest) : Two{0.f, 0.f});
        if (tid == 0) sh.count = 0;
      } else {
        int from, to;
        part_of(warp, from, to);
        all = block_add<K>(lane_sum<K, true>(sh.scale, V, cut, from, to));
      }
      target = times(all, top_p);
    }
    __syncthreads();
    const int how = sh.how;
    bool crowded = how == kCrowded;
    if (how == kFew) {
      const int n = list_from<K>(cut, least_in_bin(sh.scale, last));
      if (n <= kList) {
        __syncthreads();
        Listed mine[kListed<K>];
        rank_list<K>(n, mine);
        const int kept = keep_listed<K>(n, mine, n, cut_min, Two{0.f, 0.f}, target, err, true, loose);
        return draw_listed<K>(n, mine, kept, listed_sum(kept, Two{0.f, 0.f}), loose, u, token, logprob);
      }
      crowded = true;
      __syncthreads();
    } else if (how == kMany) {
      const Two more_part = list_border<K>(cut, first, last, sub_first, sub_last);
      if (!TWO) part = add(part, more_part);
      __syncthreads();
      if (lane == 0) sh.part2[warp] = part;
      __syncthreads();
      const int n = sh.count;
      crowded = n == 0 || n > kList;
      if (!crowded) {
        const Two ahead = warp_add(lane < K::kWarps ? sh.part2[lane] : Two{0.f, 0.f});
        Listed mine[kListed<K>];
        rank_list<K>(n, mine);
        const int kept = keep_listed<K>(n, mine, n, cut_min, ahead, target, err, false, loose);
        // the list's elements into their parts, and the cut: its last that stays, or just ahead of its first
#pragma unroll 1
        for (int e = 0; e < kListed<K>; ++e) {
          if (tid + e * K::NT >= n) break;
          if (mine[e].rank < kept) {
            sh.by_id[mine[e].rank] = mine[e].w;
            sh.list[mine[e].rank] = static_cast<Place>(id_of(mine[e].p) / K::kN / sh.per_warp);
          }
          if (mine[e].rank == 0) sh.last = cut_min.keeps(z_of(mine[e].p), id_of(mine[e].p));
          if (kept > 0 ? mine[e].rank == kept - 1 : mine[e].rank == 0)
            sh.cut = {z_of(mine[e].p), id_of(mine[e].p) - (kept > 0 ? 0 : 1)};
        }
        __syncthreads();
        cut = sh.cut;
        // (where min_p leaves out the list's first, it may leave out some of those ahead of it, too)
        summed = sh.last != 0;
        Two more{0.f, 0.f};
#pragma unroll 1
        for (int i = lane; i < kept; i += 32)
          if (static_cast<int>(sh.list[i]) == warp) more = add(more, sh.by_id[i]);
        __syncwarp();
        more = warp_add(more);
        if (lane == 0) sh.part2[warp] = add(part, more);
        __syncwarp();
      }
    }
    if (crowded) cut = select<K, true, TWO>(cut, 0, target, err, &loose);
  }
  if (!TWO && loose == INFINITY) return false;
  if (!summed) {
    if (cut_min.z > cut.z) {
      cut = cut_min;
      if (!TWO && loose > 0.f) return false;
    }
    // the sums of the warps' parts
    int from, to;
    part_of(warp, from, to);
    const Two part = sum_vectors<K, TWO>(cut, from, to);
    __syncthreads();
    if (lane == 0) sh.part2[warp] = part;
  }
  __syncthreads();
  Two part = lane < K::kWarps ? sh.part2[lane] : Two{0.f, 0.f};
  Two incl = warp_incl(part);
  const Two all = shfl(incl, 31), target = times(all, u);
  // the first part whose end passes the target
  const int w0 = first_past(incl, target, part.hi > 0.f);
  Two before = shfl(incl, (w0 + 31) & 31);
  if (w0 == 0) before = {0.f, 0.f};
  // that part of the row, cut among the warps in the same way
  int from, to;
  part_of(w0, from, to);
  const int step = ((to - from + K::kWarps - 1) / K::kWarps + 31) / 32 * 32;
  part = sum_vectors<K, TWO>(cut, min(from + warp * step, to), min(from + (warp + 1) * step, to));
  if (lane == 0) sh.part[warp] = part;
  __syncthreads();
  if (warp == 0) {
    const Scale s = sh.scale;
    part = lane < K::kWarps ? sh.part[lane] : Two{0.f, 0.f};
    incl = add(before, warp_incl(part));
    const int w1 = first_past(incl, target, part.hi > 0.f);
    if (w1 > 0) before = shfl(incl, w1 - 1);
    // and that one, 32 vectors at a time
    const int v0 = from + w1 * step, v1 = min(v0 + step, to);
    int found = -1;
    float margin = 0.f, z_found = 0.f;
#pragma unroll 1
    for (int v = v0; v < v1; v += 32) {
      // (each lane its own vector)
      Two mine{0.f, 0.f};
      if (v + lane < v1) mine = vector_sum<K, TWO>(s, V, cut, v + lane);
      __syncwarp();
      incl = add(before, warp_incl(mine));
      const unsigned has = __ballot_sync(0xffffffffu, mine.hi > 0.f);
      const unsigned past = __ballot_sync(0xffffffffu, mine.hi > 0.f && less(target, incl));
      // (the last one that has weight, as long as no later one passes the target)
      const int l = past ? __ffs(static_cast<int>(past)) - 1 : has ? 31 - __clz(static_cast<int>(has)) : -1;
      if (l >= 0) {
        Two run = shfl(incl, (l + 31) & 31);
        if (l == 0) run = before;
        // lane i: its element i
        const int id = (v + l) * K::kN + lane;
        Two w{0.f, 0.f};
        float z = -INFINITY;
        if (lane < K::kN) {
          z = element<K>(id);
          if (cut.keeps(z, id)) w = TWO ? weight2(s, sh.table, z) : Two{ex2_approx(exponent(s, z)), 0.f};
        }
        __syncwarp();
        const Two end = add(run, warp_incl(w));
        Two start = shfl(end, (lane + 31) & 31);
        if (lane == 0) start = run;
        const int e = first_past(end, target, w.hi > 0.f);
        if (lane == e && (found < 0 || !less(target, start))) {
          found = id;
          z_found = z;
          margin = minus(end, target);
          if (start.hi > 0.f || loose > 0.f) margin = fminf(margin, minus(target, start));
        }
        found = __shfl_sync(0xffffffffu, found, e);
        z_found = __shfl_sync(0xffffffffu, z_found, e);
        margin = __shfl_sync(0xffffffffu, margin, e);
      }
      before = shfl(incl, 31);
      if (past) break;
    }
    if (lane == 0) {
      sh.found = found;
      sh.logprob = logprob_of(s, z_found, all);
      sh.margin = margin;
    }
  }
  __syncthreads();
  token = sh.found;
  logprob = sh.logprob;
  const float margin = sh.margin;
  __syncthreads();
  const float off = error_of(all.hi, V) + loose;
  return TWO || (margin > 2.f * off && near_enough(off, all, logprob));
}

// The least z that `count` of the threads' two largest logits reach, or a step
// below it: at least as many of the row do.  NaN where that is not a number.
template <typename K>
__device__ __forceinline__ float reached_by(int count, float top, float z1, float z2) {
  Shared& sh = shared();
  // bins of equal width from the maximum down to the least of them
  for (int i = threadIdx.x; i < kBins; i += K::NT) sh.hist[i] = 0;
  if (threadIdx.x == 0) sh.hi = 0xffffffffu;
  __syncthreads();
  const uint32_t low = __reduce_min_sync(0xffffffffu, key_of(z2 > -INFINITY ? z2 : z1 > -INFINITY ? z1 : top));
  if ((threadIdx.x & 31) == 0) atomicMin(&sh.hi, low);
  __syncthreads();
  const float width = (0.5f * top - 0.5f * z_of(sh.hi)) / static_cast<float>(kBins - 8);
  auto bin = [&](float z) { return min(kBins - 2, static_cast<int>((0.5f * top - 0.5f * z) / width)); };
  if (!(width > 0.f)) return NAN;
  if (z1 > -INFINITY) atomicAdd(&sh.hist[bin(z1)], 1u);
  if (z2 > -INFINITY) atomicAdd(&sh.hist[bin(z2)], 1u);
  __syncthreads();
  int first, last;
  float n;
  find_bins<K>(true, 1.f, static_cast<float>(count), 0.f, first, last, n);
  if (first >= kBins || last >= kBins - 1) return NAN;
  // the least of them in those bins
  if (threadIdx.x == 0) sh.lo = 0xffffffffu;
  __syncthreads();
  uint32_t least = 0xffffffffu;
  if (z1 > -INFINITY && bin(z1) <= last) least = key_of(z1);
  if (z2 > -INFINITY && bin(z2) <= last) least = min(least, key_of(z2));
  least = __reduce_min_sync(0xffffffffu, least);
  if ((threadIdx.x & 31) == 0) atomicMin(&sh.lo, least);
  __syncthreads();
  const float z = z_of(sh.lo);
  __syncthreads();
  return z;
}

template <typename K>
__global__ void __launch_bounds__(K::NT, K::NT >= 256 ? 1024 / K::NT : 7) sample_rows(const SampleArgs a) {
  Shared& sh = shared();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long m = blockIdx.x;
  const uint4* global = reinterpret_cast<const uint4*>(static_cast<const typename K::T*>(a.logits) + m * a.ld);
  for (int i = tid; i < 64; i += K::NT) sh.table[i] = kExp2[i];
  if (tid == 0) {
    sh.bad = 0;
    sh.global = global;
    sh.V = a.V;
    sh.vecs = (a.V + K::kN - 1) / K::kN;
    sh.per_warp = ((sh.vecs + K::kWarps - 1) / K::kWarps + 31) / 32 * 32;
  }
  if (lane == 0) {
    mbar_init(smem_u32(&sh.bar[warp]), 1);
    fence_barrier_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  int from, to;  // this warp's part
  part_of(warp, from, to);
  const uint32_t bar = smem_u32(&sh.bar[warp]);
  if (K::IN_SMEM && lane == 0 && from < to) {
    mbar_arrive_expect_tx(bar, (to - from) * 16);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(row<K>() + from)),
                 "l"(global + from), "r"((to - from) * 16), "r"(bar)
                 : "memory");
  }
  __syncwarp();
  const float temperature = a.temperature ? a.temperature[m] : 1.f, top_p = a.top_p ? a.top_p[m] : 1.f,
              min_p = a.min_p ? a.min_p[m] : 0.f, u = a.uniform[m];
  const int top_k = a.top_k ? a.top_k[m] : 0;
  if (tid == K::NT - 1) {  // (one thread, while the row comes: 64-bit arithmetic is slow here)
    // 2 log2(e) / temperature
    const double counts = fmin(fmax(static_cast<double>(temperature), 0x1p-100), 0x1p100);
    const double c = 2.8853900817779268 / counts;
    sh.scale.c_hi = __double2float_rd(c * (1.0 - 0x1p-25));  // (below c)
    sh.scale.c_lo = static_cast<float>(c - sh.scale.c_hi);
    if (min_p > 0.f) sh.least = counts * log(static_cast<double>(min_p));
  }
  __syncwarp();
  // the row's maximum, and whether it has a NaN or +inf
  float top = -INFINITY, second = -INFINITY;  // this thread's largest two
  bool bad = false;
  if (K::IN_SMEM && from < to && !mbar_wait(bar, 0)) {
    record_error(a.err, kErrTimeout, kSiteSampleLoad);
    (void)mbar_wait(bar, 0);  // (the copy must not outlive the CTA)
    bad = true;
  }
#pragma unroll 2
  for (int v = from + lane; v < to; v += 32) {
    float2 z[K::kN / 2];
    vector_of<K>(v, a.V, z);
#pragma unroll
    for (int i = 0; i < K::kN; ++i) {
      second = fmaxf(second, fminf(top, at(z, i)));
      top = fmaxf(top, at(z, i));
      bad |= !(at(z, i) < INFINITY);
    }
  }
  __syncwarp();
  const float mine = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) sh.aux[warp] = top;
  if (bad) sh.bad = 1;
  __syncthreads();
  top = lane < K::kWarps ? sh.aux[lane] : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  top += 0.f;
  bad = sh.bad != 0 || top == -INFINITY;
  const bool wrong = !(temperature >= 0.f && temperature < INFINITY) || top_k < 0 || !(top_p >= 0.f) ||
                     !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f);
  int token = -1;
  float logprob = __int_as_float(0x7fffffff);
  if (wrong) {
    if (tid == 0) record_error(a.err, kErrRange, kSiteSampleRow);
  } else if (!bad && (temperature == 0.f || top_k == 1 || top_p == 0.f)) {
    // the first of the order alone
    int first = a.V;
#pragma unroll 1
    for (int v = from + lane; v < to; v += 32) {
      float2 z[K::kN / 2];
      vector_of<K>(v, a.V, z);
#pragma unroll
      for (int i = K::kN - 1; i >= 0; --i)
        if (at(z, i) == top) first = min(first, v * K::kN + i);
    }
    __syncwarp();
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.num[warp] = first;
    __syncthreads();
    first = __reduce_min_sync(0xffffffffu, lane < K::kWarps ? sh.num[lane] : a.V);
    token = first;
    logprob = 0.f;
  } else if (!bad) {
    if (tid == 0) {
      sh.scale.half_max = 0.5f * top;
      sh.cut_min = {-INFINITY, a.V - 1};
      if (min_p > 0.f) {
        // the least z with z - max >= temperature log(min_p), for the temperature that counts
        const double least = sh.least;
        float z = static_cast<float>(top + least);
        if (!(z >= -3.402823466e38f)) z = -3.402823466e38f;
        auto in = [&](float x) { return static_cast<double>(x) - top >= least; };
        // (one step at most, unless z is so small beside the maximum that the difference does not show it)
        for (int i = 0; i < 4 && z > -3.402823466e38f && in(nextafterf(z, -INFINITY)); ++i) z = nextafterf(z, -INFINITY);
        for (int i = 0; i < 4 && !in(z); ++i) z = nextafterf(z, INFINITY);
        sh.cut_min.z = z;
      }
    }
    __syncthreads();
    Cut cut{-INFINITY, a.V - 1};
    bool done = false;
    if (a.V <= kList || (top_k > 0 && top_k < a.V)) {
      const int count = top_k > 0 ? min(top_k, a.V) : a.V;
      int n = kList + 1;
      // all that can stay into the list
      if (a.V <= kList) {
        n = list_from<K>(cut, -INFINITY);
      } else if (count <= min(kList * 4 / 5, K::NT)) {
        const float least = reached_by<K>(count, top, mine, second);
        if (least == least) n = list_from<K>(cut, least);
      }
      if (n <= kList) {
        __syncthreads();
        Listed listed[kListed<K>];
        rank_list<K>(n, listed);
        const Two none{0.f, 0.f}, sum = listed_sum(min(count, n), none);
        float loose;
        const int kept = keep_listed<K>(n, listed, count, sh.cut_min, none,
                                        top_p < 1.f ? times(sum, top_p) : Two{INFINITY, 0.f}, 0.f, true, loose);
        draw_listed<K>(n, listed, kept, listed_sum(kept, none), 0.f, u, token, logprob);
        done = true;
      } else {
        __syncthreads();
        cut = select<K, false, false>(cut, count, Two{0.f, 0.f}, 0.f, nullptr);
      }
    }
    if (!done && !draw<K, false>(cut, top_p, u, token, logprob)) draw<K, true>(cut, top_p, u, token, logprob);
  }
  if (tid == 0) {
    a.tokens[m] = token;
    if (a.logprob) a.logprob[m] = logprob;
  }
}

// Threads per row: much of a row's time is latency (sums over the block, the list,
// the last steps by one warp), which other CTAs on the SM fill; so short rows take
// few threads each, and a row that fills the SM's shared memory all of them.
template <typename T, int NT, bool IN_SMEM>
cudaError_t launch_nt(const SampleArgs& a, int64_t M, size_t smem, cudaStream_t s) {
  static int configured[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(sample_rows<Kind<T, NT, IN_SMEM>>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         227 * 1024);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  return launch_pdl(sample_rows<Kind<T, NT, IN_SMEM>>, static_cast<unsigned>(M), NT, smem, s, 0, a);
}
template <typename T>
cudaError_t launch_type(const SampleArgs& a, int64_t M, cudaStream_t s) {
  const size_t need = kFixed + (static_cast<size_t>(a.V) * sizeof(T) + 15) / 16 * 16;
  const size_t own = need + 1024;  // with what the system keeps of each CTA's
  if (own <= 228 * 1024 / 5) return launch_nt<T, 128, true>(a, M, need, s);
  if (own <= 228 * 1024 / 3) return launch_nt<T, 256, true>(a, M, need, s);
  if (own <= 228 * 1024 / 2) return launch_nt<T, 512, true>(a, M, need, s);
  if (own <= 228 * 1024) return launch_nt<T, 1024, true>(a, M, need, s);
  return launch_nt<T, 1024, false>(a, M, kFixed, s);
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
