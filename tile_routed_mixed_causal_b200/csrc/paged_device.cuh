// paged_device.cuh -- pieces shared by the evicting cache's kernels: the state of a row and
// the quantisation of a page.
#pragma once

#include "tra_device.cuh"
#include "tra_launch.h"

namespace tra {

// What a row's state {n_pages, tail_len, seen, -} allows.
enum PagedRow { kRowIdle, kRowBad, kRowOk };
__device__ __forceinline__ PagedRow paged_row(int4 st, int cap) {
  if (st.x < 0) return kRowIdle;
  return st.x <= cap && st.y >= 0 && st.y < kTile ? kRowOk : kRowBad;
}

// Rounding quotients to codes without a division per value.  Adding 1.5 * 2^23 to a product
// in one fma rounds the exact product to the nearest integer, ties to even, and leaves its
// two's complement in the low bits.  Which factor rounds as the definition's division does:
//
// bf16 values (fill, and a tail that becomes a page): rne(fl32(x / s)) with s = fl32(amax / 127).
// With x = X 2^-j and amax = A (integers of 8 bits, up to a common power of two), the quotient
// y = 127 X / (A 2^j) misses a half (2 n + 1) / 2 by |254 X - A (2 n + 1) 2^j| / (A 2^(j+1)): by
// nothing, or by at least 1 / (254 X) > 2^-16 of y, while the roundings of s, of a factor near 1 / s and
// of the quotient are below 2^-20 of y.  Exact halves: 127 divides A (2 n + 1), so y is 63.5
// (|x| = amax / 2) or A is 2 * 127, where s is a power of two and every step exact.  So the
// factor is 1 / s, nudged to the side to which the definition rounds 63.5.
//
// codes of another page (evict): rne(fl32(fl32(s' c) / s)).  This quotient and c times a rounded
// s' / s (from an approximate reciprocal) differ by less than 7 * 2^-24 of the value.  So each
// code is multiplied by two factors, 2^-21 above and below: the definition's quotient lies between
// the products, and where both round to the same integer, so does it (rounding is monotone).
// Chunks with a code that straddles a half take that code's division.
constexpr float kRoundMagic = 12582912.0f;
constexpr float kAbove = 1.0f + 0x1p-21f, kBelow = 1.0f - 0x1p-21f;
// below this scale quotients of denormal values lose the bound above: always divide
constexpr float kSmallScale = 0x1p-100f;

// 1 / s to within 2^-23 of it
__device__ __forceinline__ float recip(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// low bytes of four words
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// The scale of a block of bf16 values, and the factor that rounds its quotients.
struct BlockScale {
  float s, f;
  bool divide;  // scales so small that quotients of denormal values lose the bounds above
  __device__ __forceinline__ explicit BlockScale(float amax) {
    s = __fdiv_rn(amax, 127.0f);
    divide = s < kSmallScale;
    f = recip(s);
    if ((__float_as_uint(s) & 0x007FFFFFu) == 0)
      f = __uint_as_float(0x7F000000u - __float_as_uint(s));  // a power of two: its exact reciprocal
    else
      f *= quant_code(amax * 0.5f, s, 127) == 64 ? kAbove : kBelow;
  }
};

// Codes of eight bf16 values by the definition.
static __device__ __noinline__ uint2 codes8_exact(uint4 v, float s) {
  uint2 o = make_uint2(0u, 0u);
#pragma unroll 1
  for (int j = 7; j >= 0; --j) {
    const uint32_t w = j & 4 ? (j & 2 ? v.w : v.z) : (j & 2 ? v.y : v.x);
    const uint32_t c = (uint32_t)quant_code(__uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16), s, 127) & 0xFFu;
    if (j & 4) o.y = o.y << 8 | c;
    else o.x = o.x << 8 | c;
  }
  return o;
}

// Codes of eight bf16 values (16 bytes).
__device__ __forceinline__ uint2 codes8(uint4 v, const BlockScale& b) {
  if (b.divide) return codes8_exact(v, b.s);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float2 z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    z[j] = __ffma2_rn(make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u)),
                      make_float2(b.f, b.f), make_float2(kRoundMagic, kRoundMagic));
  return make_uint2(low_bytes(z[0].x, z[0].y, z[1].x, z[1].y), low_bytes(z[2].x, z[2].y, z[3].x, z[3].y));
}

// largest |x| of eight bf16 values
__device__ __forceinline__ float amax8(uint4 v, float m) {
  auto mag = [](uint32_t w) {
    w &= 0x7FFF7FFFu;
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  };
  const __nv_bfloat162 h = __hmax2(__hmax2(mag(v.x), mag(v.y)), __hmax2(mag(v.z), mag(v.w)));
  return fmaxf(m, fmaxf(__low2float(h), __high2float(h)));
}

// The maximum of a >= 0 over a block of NT threads; red: a float per warp of shared memory.
template <int NT>
__device__ __forceinline__ float block_max(float a, float* red) {
  // (of values that are not negative: their bits are in the same order)
  a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  a = red[0];
#pragma unroll
  for (int i = 1; i < NT / 32; ++i) a = fmaxf(a, red[i]);
  return a;
}

// One page of K or V from 64 bf16 rows (NT threads): scale = fl32(amax / 127),
// code = rne(fl32(x / scale)), as everywhere in this library.  row(r): row r; codes and
// scale: the page's; red: as above, free again after the caller's next barrier.
template <int D, int NT, class Row>
__device__ __forceinline__ void quantise_page(Row row, int8_t* codes, float* scale, float* red) {
  constexpr int kChunks = D / 8, kPasses = kTile * kChunks / NT;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int f = i * NT + threadIdx.x;
    x[i] = *reinterpret_cast<const uint4*>(row(f / kChunks) + (f % kChunks) * 8);
  }
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) am = amax8(x[i], am);
  am = block_max<NT>(am, red);
  const BlockScale bs(am);
  if (threadIdx.x == 0) *scale = bs.s;
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    *reinterpret_cast<uint2*>(codes + (i * NT + threadIdx.x) * 8) = codes8(x[i], bs);
}

}  // namespace tra
