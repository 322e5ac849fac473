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

// Rounding a quotient to its code without a division per value.  y (x times the rounded
// reciprocal of the scale, or a code times a rounded ratio of scales) differs from the
// definition's quotient, whose roundings are at most three of 2^-24 each, by less than
// 127.5 * 3 * 2^-24 + 127.5 * 2^-24 < 3.1e-5; so both round to the same integer unless y
// is that near to a half, and only those values (about 1 in 10,000) take the division.
constexpr float kRoundMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer,
                                            // whose two's complement is in the low bits
constexpr float kNearHalf = 0.5f - 4e-5f;
// below this scale quotients of denormal values lose the bounds above: always divide
constexpr float kSmallScale = 7.9e-31f;     // 2^-100

// low bytes of four words
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}

// Codes of eight bf16 values (16 bytes) with scale s, r = 1 / s.
__device__ __forceinline__ uint2 codes8(uint4 v, float s, float r) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float x[8], z[8];
  float far = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    const float2 y = __fmul2_rn(make_float2(x[2 * j], x[2 * j + 1]), make_float2(r, r));
    const float2 zz = __fadd2_rn(y, make_float2(kRoundMagic, kRoundMagic));
    const float2 c = __fadd2_rn(zz, make_float2(-kRoundMagic, -kRoundMagic));
    const float2 t = __ffma2_rn(c, make_float2(-1.0f, -1.0f), y);
    z[2 * j] = zz.x;
    z[2 * j + 1] = zz.y;
    far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
  }
  if (far < kNearHalf && s >= kSmallScale)
    return make_uint2(low_bytes(z[0], z[1], z[2], z[3]), low_bytes(z[4], z[5], z[6], z[7]));
  uint32_t o[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j >> 2] |= (uint32_t)(quant_code(x[j], s, 127) & 0xFF) << ((j & 3) * 8);
  return make_uint2(o[0], o[1]);
}

// largest |x| of eight bf16 values
__device__ __forceinline__ float amax8(uint4 v, float m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
  return m;
}

// The maxima a and v over a block of 256 threads; red: 16 floats of shared memory, free to
// reuse after the caller's next barrier.
__device__ __forceinline__ float2 block_max2(float a, float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = a;
    red[8 + (threadIdx.x >> 5)] = v;
  }
  __syncthreads();
  a = red[0];
  v = red[8];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    a = fmaxf(a, red[i]);
    v = fmaxf(v, red[8 + i]);
  }
  return make_float2(a, v);
}

// One page of K and one of V from 64 bf16 rows each (256 threads): scale = fl32(amax / 127),
// code = rne(fl32(x / scale)), as everywhere in this library.  krow(r), vrow(r): row r.
template <int D, class KR, class VR>
__device__ __forceinline__ void quantise_page(const tra_paged_cache& c, int page, KR krow, VR vrow, float* red) {
  constexpr int kChunks = D / 8, kPasses = kTile * kChunks / 256;
  uint4 kx[kPasses], vx[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int f = i * 256 + threadIdx.x;
    kx[i] = *reinterpret_cast<const uint4*>(krow(f / kChunks) + (f % kChunks) * 8);
    vx[i] = *reinterpret_cast<const uint4*>(vrow(f / kChunks) + (f % kChunks) * 8);
  }
  float ka = 0.0f, va = 0.0f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    ka = amax8(kx[i], ka);
    va = amax8(vx[i], va);
  }
  const float2 am = block_max2(ka, va, red);
  const float sk = __fdiv_rn(am.x, 127.0f), sv = __fdiv_rn(am.y, 127.0f);
  const float rk = __fdiv_rn(1.0f, sk), rv = __fdiv_rn(1.0f, sv);
  if (threadIdx.x == 0) {
    c.sk[page] = sk;
    c.sv[page] = sv;
  }
  int8_t* const k8 = c.k8 + (long long)page * kTile * D;
  int8_t* const v8 = c.v8 + (long long)page * kTile * D;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int f = i * 256 + threadIdx.x;
    *reinterpret_cast<uint2*>(k8 + f * 8) = codes8(kx[i], sk, rk);
    *reinterpret_cast<uint2*>(v8 + f * 8) = codes8(vx[i], sv, rv);
  }
}

}  // namespace tra
