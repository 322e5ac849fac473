// paged_cut.cu -- filling the evicting cache from a prompt and shrinking it: both choose a
// row's survivors by accumulated weight and write them as pages of 64 quantised tokens.
//
// Selection, one CTA of 1024 threads per (sequence, KV head): the weights' ordered bits are
// staged once in shared memory, protected tokens as the largest; a radix select (three digits
// of 11, 11 and 10 bits) finds the last key that survives, and one ascending pass writes the
// survivors' indices at their ranks, ties taken in order.  Bound by latency: a dozen
// block-wide steps, so it writes nothing but the indices.  32K tokens: 22 us, 26 us where the
// weights of all heads lie side by side (fill); 4K: 6 us.  One more CTA per sequence checks its
// page numbers meanwhile and says what becomes of the row.
//
// Pages, one CTA per (up to four pages, K or V, KV head, sequence): 64 gathered rows are held in
// registers while their maximum is reduced, then written as codes, the next page's rows
// already on their way; the K part moves the tokens' weights, the V part their positions.
// One read and one write of what survives: bound by memory.  (Survivors are single rows of
// d values anywhere in the source, 64 to 256 bytes each: every access is whole sectors.)
// 16 x 32K tokens: fill to 8K per head 141 us (5.7 TB/s), evict to 16K 276 us (4.0 TB/s; 11
// instructions per code bound it).  K and V apart, and 32 values or 64 codes per thread, leave
// room for enough CTAs; half or double the threads cost evict 20 %.
//
// A row that is cut in place gets its weights and positions through the workspace and a
// third kernel, since pages are written in any order.
#include <cuda_fp16.h>

#include "launch_ex.cuh"
#include "paged_device.cuh"

namespace tra {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSpan = 48 * 1024;      // tokens ranked at a time; keys that fit shared memory (192 KB)
constexpr int kSpanChunks = kSpan / (4 * kSelThreads);
constexpr uint32_t kKeepKey = 0xFFFFFFFFu;  // above every finite weight's key

// Monotone map of a float's bits to unsigned order (-0 as +0); finite values map above 0.
__device__ __forceinline__ uint32_t order_of(float f) {
  uint32_t u = __float_as_uint(f);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block; the total in `all`.  tmp: 33 words, and two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* tmp, uint32_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const uint32_t w = tmp[lane];
    uint32_t t = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    tmp[lane] = t - w;
    if (lane == 31) tmp[32] = t;
  }
  __syncthreads();
  all = tmp[32];
  return tmp[warp] + s - v;
}

// Evict: the row is to be cut; and has the free pages for it.
__device__ __forceinline__ bool cut_due(const PagedCutParams& p, int4 st) {
  return paged_row(st, p.c.cap) == kRowOk && st.x > p.keep && st.x * kTile + st.y >= p.least;
}
__device__ __forceinline__ bool cut_fits(const PagedCutParams& p, int4 st) {
  return cut_due(p, st) && st.x <= p.c.cap - p.keep;
}

// What becomes of row b, for the kernels behind the selection: the CTA before those of its heads.
// Where one of the page numbers that the row's pages would be read by and written to is out of
// range, in any head, the whole row stays.  (Fill of one 8K prompt: 11.3 us with and without the check,
// 11.6 with this CTA behind the heads', 12.1 checked by the selections themselves and joined by the
// pages' CTAs.)
template <bool FILL>
__device__ __forceinline__ void check_row(const PagedCutParams& p, int b) {
  const tra_paged_cache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int4 st;      // as paged_write_kernel takes it
  int used;     // table entries of each head
  if (FILL) {
    const int total = __ldg(p.cu + b + 1) - __ldg(p.cu + b);
    used = min(total / kTile, p.keep);
    st = make_int4(used, total % kTile, total, 1);
  } else {
    const int4 s = reinterpret_cast<const int4*>(c.state)[b];
    const PagedRow kind = paged_row(s, c.cap);
    const bool cut = cut_fits(p, s);
    st = make_int4(s.x, s.y, kind == kRowOk, cut);
    used = cut ? s.x + p.keep : 0;
    if (threadIdx.x == 0) {
      if (kind == kRowBad) atomicOr(p.status, TRA_DEV_BAD_CACHE);
      if (cut_due(p, s) && !cut) atomicOr(p.status, TRA_DEV_CACHE_FULL);
    }
  }
  bool bad = false;
  const int parts = max(1, kSelThreads / 32 / c.Hkv);  // warps of a head
  for (int u = warp; u < c.Hkv * parts; u += kSelThreads / 32) {
    const int32_t* const table = c.table + ((long long)b * c.Hkv + u / parts) * c.cap;
#pragma unroll 4
    for (int k = u % parts * 32 + lane; k < used; k += 32 * parts) bad |= table[k] < 0 || table[k] >= c.n_pool;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    if (bad) atomicOr(p.status, TRA_DEV_BAD_CACHE);
    st.w = st.w && !bad;
    p.ws_state[b] = st;
  }
}

template <bool FILL>
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const PagedCutParams p, int stage) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t tmp[33];
  __shared__ uint2 warp_sum[kSpanChunks * 32 + 1];
  __shared__ uint32_t s_bin, s_want;
  grid_release();
  const int g = (int)blockIdx.x - 1, b = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const tra_paged_cache& c = p.c;
  if (g < 0) {
    check_row<FILL>(p, b);
    return;
  }
  const int row = b * c.Hkv + g;
  const long long row64 = (long long)row * (c.cap + 1) * kTile;

  // tokens to choose among (body), pages after the call (n), all tokens (total)
  int body, n, from = 0, total = 0;
  if (FILL) {
    from = __ldg(p.cu + b);
    total = __ldg(p.cu + b + 1) - from;
    body = total / kTile * kTile;
    n = min(body / kTile, p.keep);
  } else {
    const int4 st = reinterpret_cast<const int4*>(c.state)[b];
    if (!cut_fits(p, st)) return;
    body = st.x * kTile;
    n = p.keep;
    total = body + st.y;
  }
  const int m = n * kTile;
  // the tokens from `first` on survive whatever their weight
  int first = !FILL || p.imp ? min(max(total - p.recent, body - m), body) : body - m;
  if (m == body) first = 0;
  int32_t* const out = p.ws_src + (long long)row * c.cap * kTile;
  if (body - first == m) {
    for (int i = t; i < m; i += kSelThreads) out[i] = first + i;
    return;
  }

  const float* const w_row = FILL ? p.imp + (long long)from * c.Hkv + g : c.weight + row64;
  const long long w_step = FILL ? c.Hkv : 1;
  auto load_key = [&](int j) -> uint32_t { return j < first ? order_of(w_row[j * w_step]) : kKeepKey; };
  const bool staged = body <= stage;  // (a multiple of 64)
  auto key4 = [&](int j) -> uint4 {   // of tokens j .. j + 3, j a multiple of 4
    if (j >= body) return make_uint4(0, 0, 0, 0);
    if (staged) return *reinterpret_cast<const uint4*>(keys + j);
    return make_uint4(load_key(j), load_key(j + 1), load_key(j + 2), load_key(j + 3));
  };
  hist[t] = 0;
  hist[t + kSelThreads] = 0;
  __syncthreads();
  if (staged) {
    if (FILL) {
#pragma unroll 8
      for (int j = t; j < body; j += kSelThreads) {
        const uint32_t k = load_key(j);
        keys[j] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
    } else {  // a row's weights start on a 256-byte boundary
#pragma unroll 4
      for (int j = 4 * t; j < body; j += 4 * kSelThreads) {
        const float4 v = *reinterpret_cast<const float4*>(w_row + j);
        uint4 k = make_uint4(order_of(v.x), order_of(v.y), order_of(v.z), order_of(v.w));
        if (j + 3 >= first) {
          if (j >= first) k.x = kKeepKey;
          if (j + 1 >= first) k.y = kKeepKey;
          if (j + 2 >= first) k.z = kKeepKey;
          k.w = kKeepKey;
        }
        *reinterpret_cast<uint4*>(keys + j) = k;
        atomicAdd(&hist[k.x >> 21], 1u);
        atomicAdd(&hist[k.y >> 21], 1u);
        atomicAdd(&hist[k.z >> 21], 1u);
        atomicAdd(&hist[k.w >> 21], 1u);
      }
    }
  } else {
    for (int j = t; j < body; j += kSelThreads) atomicAdd(&hist[load_key(j) >> 21], 1u);
  }

  // ---- the m-th largest key, and how many of the keys equal to it survive
  uint32_t kth = 0, need = (uint32_t)m;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    if (pass > 0) {
      hist[t] = 0;
      hist[t + kSelThreads] = 0;
      __syncthreads();
      for (int j = 4 * t; j < body; j += 4 * kSelThreads) {
        const uint4 k4 = key4(j);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if ((k[y] >> (shift + bits)) == kth) atomicAdd(&hist[(k[y] >> shift) & ((1u << bits) - 1u)], 1u);
      }
    }
    __syncthreads();
    // from the top: thread t has bins 2047 - 2t and 2046 - 2t
    const uint32_t h0 = hist[2047 - 2 * t], h1 = hist[2046 - 2 * t];
    uint32_t sum;
    const uint32_t above = block_scan(h0 + h1, tmp, sum);
    if (above < need && need <= above + h0 + h1) {
      const bool second = need > above + h0;
      s_bin = 2047 - 2 * t - second;
      s_want = need - above - (second ? h0 : 0);
    }
    __syncthreads();
    kth = (kth << bits) | s_bin;
    need = s_want;
  }
  const uint32_t ties = need;

  // ---- ranks, a span at a time: per-warp counts of keys above and equal, their prefix over
  // the span, then each survivor's index at its rank
  uint32_t above0 = 0, equal0 = 0;
  for (int s0 = 0; s0 < body; s0 += kSpan) {
    const int chunks = (min(kSpan, body - s0) + 4 * kSelThreads - 1) / (4 * kSelThreads);
    for (int i = 0; i < chunks; ++i) {
      const uint4 k = key4(s0 + (i * kSelThreads + t) * 4);
      const uint32_t a = (k.x > kth) + (k.y > kth) + (k.z > kth) + (k.w > kth);
      const uint32_t e = (k.x == kth) + (k.y == kth) + (k.z == kth) + (k.w == kth);
      const uint32_t both = __reduce_add_sync(0xffffffffu, a << 16 | e);
      if (lane == 0) warp_sum[i * 32 + warp] = make_uint2(both >> 16, both & 0xFFFFu);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefix in place: lane l has entries l * chunks ..
      uint2 own = make_uint2(0, 0);
      for (int i = 0; i < chunks; ++i) {
        const uint2 v = warp_sum[lane * chunks + i];
        own.x += v.x;
        own.y += v.y;
      }
      uint2 run = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, run.x, o), y = __shfl_up_sync(0xffffffffu, run.y, o);
        if (lane >= o) {
          run.x += x;
          run.y += y;
        }
      }
      if (lane == 31) warp_sum[kSpanChunks * 32] = run;
      run.x -= own.x;
      run.y -= own.y;
      for (int i = 0; i < chunks; ++i) {
        const uint2 v = warp_sum[lane * chunks + i];
        warp_sum[lane * chunks + i] = run;
        run.x += v.x;
        run.y += v.y;
      }
    }
    __syncthreads();
    for (int i = 0; i < chunks; ++i) {
      const int j = s0 + (i * kSelThreads + t) * 4;
      const uint4 k4 = key4(j);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
      uint32_t both = 0;
#pragma unroll
      for (int y = 0; y < 4; ++y) both += k[y] > kth ? 0x10000u : k[y] == kth ? 1u : 0u;
      uint32_t pre = both;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += u;
      }
      pre -= both;
      const uint2 w = warp_sum[i * 32 + warp];
      uint32_t a = above0 + w.x + (pre >> 16), e = equal0 + w.y + (pre & 0xFFFFu);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const bool gt = k[y] > kth, eq = k[y] == kth;
        if (gt || (eq && e < ties)) out[a + min(e, ties)] = j + y;
        a += gt;
        e += eq;
      }
    }
    const uint2 all = warp_sum[kSpanChunks * 32];
    above0 += all.x;
    equal0 += all.y;
    __syncthreads();
  }
}

// x = code * s of a source page: sixteen codes as floats
__device__ __forceinline__ void floats16(uint4 v, float (&f)[16]) {
  const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the biased byte as the low bits of 2^23, then the bias off: exact
    const float b0 = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7440));
    const float b1 = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7441));
    const float b2 = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7442));
    const float b3 = __uint_as_float(__byte_perm(w[i], 0x4B000000u, 0x7443));
    const float2 off = make_float2(-8388736.0f, -8388736.0f);
    const float2 lo = __fadd2_rn(make_float2(b0, b1), off), hi = __fadd2_rn(make_float2(b2, b3), off);
    f[4 * i] = lo.x;
    f[4 * i + 1] = lo.y;
    f[4 * i + 2] = hi.x;
    f[4 * i + 3] = hi.y;
  }
}

// The largest and the smallest biased code seen so far, in 16-bit pairs.
struct CodeRange {
  uint32_t hi, lo;
  __device__ __forceinline__ void reset() {
    hi = 0u;
    lo = 0x00FF00FFu;
  }
  __device__ __forceinline__ void add(uint4 v) {
    const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t even = w[i] & 0x00FF00FFu, odd = __byte_perm(w[i], 0u, 0x4341);
      hi = __vimax3_u16x2(hi, even, odd);
      lo = __vimin3_u16x2(lo, even, odd);
    }
  }
  __device__ __forceinline__ float largest() const {  // |code|
    const int h = max(hi & 0xFFFFu, hi >> 16), l = min(lo & 0xFFFFu, lo >> 16);
    return (float)max(h - 128, 128 - l);
  }
};

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

// Rare, and kept out of the loops: inlined and unrolled, the divisions overflowed the
// instruction cache (evict of 16 x 32K: 570 us).
__device__ __noinline__ uint32_t code_exact(float s, float f, float sn) {
  return (uint32_t)quant_code(__fmul_rn(s, f), sn, 127);
}

// recode16 where some values straddle a half: those by the definition.
__device__ __noinline__ uint4 recode16_exact(uint4 v, float s, float sn, float fa, float fb) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = __uint_as_float(__byte_perm(w[i] ^ 0x80808080u, 0x4B000000u, 0x7440 + j)) - 8388736.0f;
      const float za = fmaf(f, fa, kRoundMagic), zb = fmaf(f, fb, kRoundMagic);
      uint32_t c = __float_as_uint(za);
      if (!(za == zb) || sn < kSmallScale) c = code_exact(s, f, sn);
      o = j == 0 ? c & 0xFFu : __byte_perm(o, c, j == 1 ? 0x3240 : j == 2 ? 0x3410 : 0x4210);
    }
    w[i] = o;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of fl32(s * code) for the new scale sn; fa, fb: s / sn, above and below.
__device__ __forceinline__ uint4 recode16(uint4 v, float s, float sn, float fa, float fb) {
  float f[16], z[16];
  floats16(v, f);
  if (round_codes<16>(f, fa, fb, z) == 0.0f && sn >= kSmallScale)
    return make_uint4(low_bytes(z[0], z[1], z[2], z[3]), low_bytes(z[4], z[5], z[6], z[7]),
                      low_bytes(z[8], z[9], z[10], z[11]), low_bytes(z[12], z[13], z[14], z[15]));
  return recode16_exact(v, s, sn, fa, fb);
}

// What a thread holds of a page of K or V: 16-byte chunks of gathered rows, per two of which
// (evict) one scale, and a token's weight or position.
template <int D, bool FILL>
struct PageCfg {
  static constexpr int kThreads = FILL ? 256 : 128;            // 32 bf16 values or 64 codes each
  static constexpr int kChunks = FILL ? D / 8 : D / 16;        // of a row
  static constexpr int kVec = kTile * kChunks / kThreads;
  static constexpr int kRowThreads = FILL ? kChunks : 4;       // threads that share a row
  static constexpr int kRowStep = kThreads / kRowThreads;      // rows a thread's chunks are apart
  static constexpr int kRowsEach = kTile / kRowStep;           // rows per thread
  static constexpr int kPerRow = kVec / kRowsEach;             // chunks of each
};

template <int D, bool FILL>
struct PageRows {
  using C = PageCfg<D, FILL>;
  uint4 v[C::kVec];
  float s[FILL ? 1 : C::kRowsEach];
  uint32_t side;  // weight bits or position of token t of the page (t < 64)
  int page;       // destination
};

// The K (V) part of pages i0 .. i0 + per - 1 of one row.  While a page's values are reduced and
// written the next page's rows are on their way.
template <int D, bool FILL>
__global__ void __launch_bounds__(PageCfg<D, FILL>::kThreads, FILL ? 4 : 7)
    paged_write_kernel(const PagedCutParams p, int per, int groups) {
  using C = PageCfg<D, FILL>;
  constexpr int NT = C::kThreads;
  __shared__ float red[2][NT / 32];
  const int is_v = blockIdx.x & 1, grp_i = blockIdx.x >> 1, g = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const tra_paged_cache& c = p.c;
  grid_release();
  grid_wait();
  const int4 st = p.ws_state[b];  // fill {pages, tail, seen, goes}, evict {pages before, tail, valid, cut}
  const int row = b * c.Hkv + g;
  const long long row64 = (long long)row * (c.cap + 1) * kTile;
  const int32_t* const table = c.table + (long long)row * c.cap;
  float* const w_out = p.weight_out + row64;
  int32_t* const p_out = p.pos_out + row64;

  if (grp_i == groups) {  // what lies behind the pages
    const int4 old = reinterpret_cast<const int4*>(c.state)[b];
    if (FILL) {  // the tail's rows, weights and positions
      if (!st.w) return;
      const int from = __ldg(p.cu + b) + st.z - st.y;
      const uint16_t* const x = is_v ? p.v : p.k;
      uint16_t* const tail = is_v ? c.v_tail : c.k_tail;
      for (int f = t; f < st.y * (D / 8); f += NT) {
        const int r = f / (D / 8), ch = f % (D / 8) * 8;
        *reinterpret_cast<uint4*>(tail + ((long long)row * kTile + r) * D + ch) =
            *reinterpret_cast<const uint4*>(x + ((long long)(from + r) * c.Hkv + g) * D + ch);
      }
      if (t < st.y) {
        if (is_v) p_out[st.x * kTile + t] = st.z - st.y + t;
        else w_out[st.x * kTile + t] = p.imp ? p.imp[(long long)(from + t) * c.Hkv + g] : 0.0f;
      }
      if (g == 0 && !is_v && t == 0) reinterpret_cast<int4*>(p.state_out)[b] = make_int4(st.x, st.y, st.z, 0);
      return;
    }
    // evict: tail weights and positions; a row that stays moves over whole, where that is elsewhere
    const int n = st.x, keep = p.keep, m0 = st.w ? n * kTile : 0, d0 = st.w ? keep * kTile : 0;
    const int cnt = st.w ? st.y : (st.z && !p.in_place) ? n * kTile + st.y : 0;
    for (int k = t; k < cnt; k += NT) {
      if (is_v) p_out[d0 + k] = c.pos[row64 + m0 + k];
      else w_out[d0 + k] = c.weight[row64 + m0 + k];
    }
    if (is_v && !p.in_place)  // the table turns by the new pages
      for (int k = t; k < c.cap; k += NT)
        p.table_out[(long long)row * c.cap + k] =
            table[!st.w || k >= n + keep ? k : k < keep ? n + k : k - keep];
    if (g == 0 && !is_v && t == 0)
      reinterpret_cast<int4*>(p.state_out)[b] = make_int4(st.w ? keep : old.x, old.y, old.z, old.w);
    return;
  }
  const int i0 = grp_i * per, i1 = min(i0 + per, !st.w ? 0 : FILL ? st.x : p.keep);
  if (i0 >= i1) return;
  int8_t* const codes = is_v ? c.v8 : c.k8;
  float* const scales = is_v ? c.sv : c.sk;
  const long long from = FILL ? __ldg(p.cu + b) : 0;
  const int r0 = t / C::kRowThreads, ch0 = t % C::kRowThreads;

  // the thread's survivors of page i: their rows' sources and, for t < 64, token t
  auto sources = [&](int i, int (&src)[C::kRowsEach], int& tok) {
    const int32_t* const s = p.ws_src + ((long long)row * c.cap + i) * kTile;
#pragma unroll
    for (int y = 0; y < C::kRowsEach; ++y) src[y] = s[r0 + y * C::kRowStep];
    tok = t < kTile ? s[t] : 0;
    if (!FILL) {  // evict: the rows of the codes
#pragma unroll
      for (int y = 0; y < C::kRowsEach; ++y) src[y] = table[src[y] / kTile] * kTile + src[y] % kTile;
    }
  };
  auto fetch = [&](int i, const int (&src)[C::kRowsEach], int tok, PageRows<D, FILL>& x) {
#pragma unroll
    for (int y = 0; y < C::kRowsEach; ++y) {
      if constexpr (FILL) {
        const uint16_t* const a = (is_v ? p.v : p.k) + ((from + src[y]) * c.Hkv + g) * D;
#pragma unroll
        for (int k = 0; k < C::kPerRow; ++k)
          x.v[y * C::kPerRow + k] = *reinterpret_cast<const uint4*>(a + (ch0 + k * C::kRowThreads) * 8);
      } else {
        const int8_t* const a = codes + (long long)src[y] * D;
#pragma unroll
        for (int k = 0; k < C::kPerRow; ++k)
          x.v[y * C::kPerRow + k] = *reinterpret_cast<const uint4*>(a + (ch0 + k * C::kRowThreads) * 16);
        x.s[y] = scales[src[y] / kTile];
      }
    }
    if (t < kTile) {
      if (is_v) x.side = FILL ? tok : c.pos[row64 + tok];
      else x.side = __float_as_uint(FILL ? (p.imp ? p.imp[(from + tok) * c.Hkv + g] : 0.0f) : c.weight[row64 + tok]);
    }
    x.page = table[(FILL ? 0 : st.x) + i];
  };
  auto write = [&](int i, const PageRows<D, FILL>& x, float* r) {
    if (t < kTile) {
      if (is_v) p_out[i * kTile + t] = (int)x.side;
      else w_out[i * kTile + t] = __uint_as_float(x.side);
    }
    float am = 0.0f;
    if constexpr (FILL) {
#pragma unroll
      for (int k = 0; k < C::kVec; ++k) am = amax8(x.v[k], am);
    } else {  // fl32(s * code) grows with |code|: a row's largest is s times its largest code
#pragma unroll
      for (int y = 0; y < C::kRowsEach; ++y) {
        CodeRange range;
        range.reset();
#pragma unroll
        for (int k = 0; k < C::kPerRow; ++k) range.add(x.v[y * C::kPerRow + k]);
        am = fmaxf(am, __fmul_rn(x.s[y], range.largest()));
      }
    }
    am = block_max<NT>(am, r);
    int8_t* const dst = codes + (long long)x.page * kTile * D;
    if constexpr (FILL) {
      const BlockScale bs(am);
      if (t == 0) scales[x.page] = bs.s;
#pragma unroll
      for (int y = 0; y < C::kRowsEach; ++y)
#pragma unroll
        for (int k = 0; k < C::kPerRow; ++k)
          *reinterpret_cast<uint2*>(dst + (r0 + y * C::kRowStep) * D + (ch0 + k * C::kRowThreads) * 8) =
              codes8(x.v[y * C::kPerRow + k], bs);
    } else {
      const float sn = __fdiv_rn(am, 127.0f), inv = recip(sn);
      if (t == 0) scales[x.page] = sn;
#pragma unroll
      for (int y = 0; y < C::kRowsEach; ++y) {
        const float f = x.s[y] * inv;
        const float fa = f * kAbove, fb = f * kBelow;
#pragma unroll
        for (int k = 0; k < C::kPerRow; ++k)
          *reinterpret_cast<uint4*>(dst + (r0 + y * C::kRowStep) * D + (ch0 + k * C::kRowThreads) * 16) =
              recode16(x.v[y * C::kPerRow + k], x.s[y], sn, fa, fb);
      }
    }
  };

  int src[C::kRowsEach], tok;
  PageRows<D, FILL> x0, x1;
  sources(i0, src, tok);
  fetch(i0, src, tok, x0);
  if (i0 + 1 < i1) sources(i0 + 1, src, tok);
  for (int i = i0; i < i1; i += 2) {
    if (i + 1 < i1) fetch(i + 1, src, tok, x1);
    if (i + 2 < i1) sources(i + 2, src, tok);
    write(i, x0, red[0]);
    if (i + 1 >= i1) break;
    if (i + 2 < i1) fetch(i + 2, src, tok, x0);
    if (i + 3 < i1) sources(i + 3, src, tok);
    write(i + 1, x1, red[1]);
  }
}

// In place: the weights and positions of a row that was cut come back from the workspace,
// and its table turns (the old pages move up by `keep`, the last ones first).
__global__ void __launch_bounds__(kSelThreads) paged_settle_kernel(const PagedCutParams p) {
  const int g = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  const tra_paged_cache& c = p.c;
  grid_wait();
  const int4 st = p.ws_state[b];
  if (!st.w) return;
  const int row = b * c.Hkv + g, keep = p.keep, n = st.x;
  const long long row64 = (long long)row * (c.cap + 1) * kTile;
  for (int k = t; k < keep * kTile + st.y; k += kSelThreads) {
    c.weight[row64 + k] = p.weight_out[row64 + k];
    c.pos[row64 + k] = p.pos_out[row64 + k];
  }
  int32_t* const table = c.table + (long long)row * c.cap;
  int32_t* const fresh = p.ws_dst + (long long)row * c.cap;
  for (int k = t; k < keep; k += kSelThreads) fresh[k] = table[n + k];
  __syncthreads();
  for (int hi = n; hi > 0; hi -= kSelThreads) {
    const int k = hi - 1 - t;
    const int page = k >= 0 ? table[k] : 0;
    __syncthreads();
    if (k >= 0) table[keep + k] = page;
    __syncthreads();
  }
  for (int k = t; k < keep; k += kSelThreads) table[k] = fresh[k];
}

template <bool FILL>
cudaError_t launch_cut(const PagedCutParams& p, cudaStream_t s) {
  const tra_paged_cache& c = p.c;
  const int stage = p.nmax < kSpan ? p.nmax : kSpan;
  const size_t smem = ((size_t)stage * 4 + 15) & ~(size_t)15;
  static SmemLimit limit;
  cudaError_t e = limit.raise(paged_select_kernel<FILL>, kSpan * 4);
  if (e != cudaSuccess) return e;
  e = launch_ex(paged_select_kernel<FILL>, dim3(c.Hkv + 1, c.B), kSelThreads, smem, s, 0, false, p, stage);
  if (e != cudaSuccess) return e;
  // one page per CTA until every SM has its fill of them, then up to four
  const long long ctas = 2ll * p.keep * c.Hkv * c.B;
  const int per = ctas >= 4 * 148 * 8 ? 4 : ctas >= 2 * 148 * 8 ? 2 : 1;
  const int groups = (p.keep + per - 1) / per;
  const dim3 grid(2 * (groups + 1), c.Hkv, c.B);
  e = c.d == 128 ? launch_ex(paged_write_kernel<128, FILL>, grid, PageCfg<128, FILL>::kThreads, 0, s, 0, true, p, per, groups)
                 : launch_ex(paged_write_kernel<64, FILL>, grid, PageCfg<64, FILL>::kThreads, 0, s, 0, true, p, per, groups);
  if (e != cudaSuccess || !p.in_place) return e;
  return launch_ex(paged_settle_kernel, dim3(c.Hkv, c.B), kSelThreads, 0, s, 0, true, p);
}

}  // namespace

cudaError_t launch_paged_fill(const PagedCutParams& p, cudaStream_t s) { return launch_cut<true>(p, s); }
cudaError_t launch_paged_evict(const PagedCutParams& p, cudaStream_t s) { return launch_cut<false>(p, s); }

}  // namespace tra
