// Pieces of the attention kernels over a paged key-value cache.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace gpt2 {

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

// fp16 probabilities are carried 2^12 times larger: their smallest step is then
// 2^-36 of the row's largest and not 2^-24.
template <typename T16>
constexpr float kShift = std::is_same<T16, __half>::value ? 12.f : 0.f;

// Adds a piece (its 4 values x, its m and l) to (acc, M, L).  KEEP_INF: an infinity stays
// one however little it counts: 2^-149 times at least, with which finite values add
// 2^-21 at most.
template <bool KEEP_INF = false>
__device__ __forceinline__ void merge(float4& acc, float& M, float& L, const float4& x, const float2& ml) {
  if (ml.y == 0.f) return;  // nothing in it but scores of -inf
  const float mn = fmaxf(M, ml.x);
  float c0 = M == mn ? 1.f : ex2_approx(M - mn), c1 = ml.x == mn ? 1.f : ex2_approx(ml.x - mn);
  if constexpr (KEEP_INF) {
    c0 = __int_as_float(max(__float_as_int(c0), 1));
    c1 = __int_as_float(max(__float_as_int(c1), 1));
  }
  M = mn;
  L = L * c0 + ml.y * c1;
  acc.x = acc.x * c0 + x.x * c1;
  acc.y = acc.y * c0 + x.y * c1;
  acc.z = acc.z * c0 + x.z * c1;
  acc.w = acc.w * c0 + x.w * c1;
}

}  // namespace gpt2
