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

// Rounding a quotient to its code without a division per value.  The definition's quotient
// fl32(x / s) (evict: fl32(fl32(s' code) / s)) and a value times a rounded factor 1 / s
// (s' / s, from an approximate reciprocal) differ by less than 7 * 2^-24 of the value.  So each value is
// multiplied by two factors, 2^-21 above and below the rounded one: the definition's
// quotient lies between the products, and where both round to the same integer, so does
// it (rounding is monotone).  Values that straddle a half take the division: about one in
// 25,000, and the exact halves (half the block's largest value: 63.5).
// Adding 1.5 * 2^23 in the same fma rounds the exact product to the nearest integer, ties
// to even, and leaves its two's complement in the low bits.
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

// N values times the factor one side (fa) and the other (fb): fa's rounded products in the
// low bits of z; returns how many values' two products differ.
template <int N>
__device__ __forceinline__ float round_codes(const float (&x)[N], float fa, float fb, float (&z)[N]) {
  float2 apart = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const float2 v = make_float2(x[j], x[j + 1]);
    const float2 za = __ffma2_rn(v, make_float2(fa, fa), make_float2(kRoundMagic, kRoundMagic));
    const float2 zb = __ffma2_rn(v, make_float2(-fb, -fb), make_float2(-kRoundMagic, -kRoundMagic));
    const float2 e = __fadd2_rn(za, zb);  // 0 or +-1
    apart = __ffma2_rn(e, e, apart);
    z[j] = za.x;
    z[j + 1] = za.y;
  }
  return apart.x + apart.y;
}

// The scale of a block of bf16 values and the factors that round its quotients: 63.5, the one
// quotient that bf16 values hit often (any |x| that is half the largest), is divided once, and
// `fa` is the side that rounds it as the definition does.
struct BlockScale {
  float s, fa, fb;
  uint32_t half;  // half the largest value, twice
  __device__ __forceinline__ explicit BlockScale(float amax) {
    s = __fdiv_rn(amax, 127.0f);
    const float r = recip(s);
    const bool up = quant_code(amax * 0.5f, s, 127) == 64;
    fa = r * (up ? kAbove : kBelow);
    fb = r * (up ? kBelow : kAbove);
    half = (__float_as_uint(amax * 0.5f) >> 16) * 0x10001u;
  }
};

// Codes of eight bf16 values by the definition.  Rare, and kept out of the loops: inlined and
// unrolled, the divisions overflowed the instruction cache (evict of 16 x 32K: 570 us).
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
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8], z[8];
  __nv_bfloat162 halves = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    const uint32_t mag = w[j] & 0x7FFF7FFFu;
    halves = __hadd2(halves, __heq2(*reinterpret_cast<const __nv_bfloat162*>(&mag),
                                    *reinterpret_cast<const __nv_bfloat162*>(&b.half)));
  }
  const float apart = round_codes<8>(x, b.fa, b.fb, z);
  // (a NaN, from a scale of zero, compares unequal)
  if (apart == __low2float(halves) + __high2float(halves) && b.s >= kSmallScale)
    return make_uint2(low_bytes(z[0], z[1], z[2], z[3]), low_bytes(z[4], z[5], z[6], z[7]));
  return codes8_exact(v, b.s);
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
