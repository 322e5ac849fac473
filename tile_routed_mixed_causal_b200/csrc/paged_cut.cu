// paged_cut.cu -- filling the evicting cache from a prompt and shrinking it: both choose a
// row's survivors by accumulated weight and write them as pages of 64 quantised tokens.
//
// Selection, one CTA of 1024 threads per (sequence, KV head): the weights' ordered bits are
// staged once in shared memory; a radix select (three digits of 11, 11 and 10 bits) finds
// the want-th largest, and one ascending pass of 4096 tokens at a time writes the survivors'
// source rows, weights and positions at their ranks, ties taken in order.  Every chunk is
// read by the whole block before any of it is written, and a survivor never moves up, so a
// row can be cut in place.  Bound by latency: some ten block-wide steps.
//
// Pages, one CTA of 256 threads per (page, KV head, sequence): 64 gathered rows of K and of
// V are held in registers while their maxima are reduced, then written as codes: one read
// and one write of what survives, bound by memory.  (Survivors are single rows of d values
// anywhere in the source, 128 to 256 bytes each: every access is whole sectors.)
#include "paged_device.cuh"

namespace tra {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kChunkTok = 4 * kSelThreads;
constexpr int kStageMax = 48 * 1024;  // keys held in shared memory (192 KB)

// Monotone map of a float's bits to unsigned order (-0 as +0), and back.
__device__ __forceinline__ uint32_t order_of(float f) {
  uint32_t u = __float_as_uint(f);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
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

template <bool FILL>
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const PagedCutParams p, int stage) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t tmp[33];
  __shared__ uint32_t s_bin, s_want;
  const int g = blockIdx.x, b = blockIdx.y, t = threadIdx.x;
  const tra_paged_cache& c = p.c;
  const int row = b * c.Hkv + g;
  const long long row64 = (long long)row * (c.cap + 1) * kTile;
  int32_t* const table = c.table + (long long)row * c.cap;
  int32_t* const table_out = p.table_out + (long long)row * c.cap;

  // tokens to choose among (body), tail behind them, pages after the call (n)
  int body, tail, n, from = 0, total = 0;
  if (FILL) {
    from = __ldg(p.cu + b);
    total = __ldg(p.cu + b + 1) - from;
    body = total / kTile * kTile;
    tail = total - body;
    n = min(body / kTile, p.keep);
    if (g == 0 && t == 0) p.ws_state[b] = make_int4(n, tail, total, 1);
  } else {
    const int4 st = reinterpret_cast<const int4*>(c.state)[b];
    const PagedRow kind = paged_row(st, c.cap);
    const bool full = kind == kRowOk && st.x > p.keep && st.x > c.cap - p.keep;
    const bool cut = kind == kRowOk && st.x > p.keep && !full;
    if (g == 0 && t == 0) {
      p.ws_state[b] = make_int4(p.keep, st.y, st.z, cut);
      if (kind == kRowBad) atomicOr(p.status, TRA_DEV_BAD_CACHE);
      if (full) atomicOr(p.status, TRA_DEV_CACHE_FULL);
    }
    if (!cut) {  // the row stays: into the output arrays as it is
      if (table_out != table) {
        for (int i = t; i < c.cap; i += kSelThreads) table_out[i] = table[i];
        const int m = kind == kRowOk ? st.x * kTile + st.y : 0;
        for (int i = t; i < m; i += kSelThreads) {
          p.weight_out[row64 + i] = c.weight[row64 + i];
          p.pos_out[row64 + i] = c.pos[row64 + i];
        }
      }
      return;
    }
    body = st.x * kTile;
    tail = st.y;
    n = p.keep;
    total = body + tail;
  }
  const int m = n * kTile;
  // tokens from `first` on are kept; `want` more among those before it
  const bool ranked = !FILL || p.imp != nullptr;
  int first = ranked ? max(total - p.recent, body - m) : body - m;
  first = min(first, body);
  const int want = m - (body - first);

  auto weight_at = [&](int j) -> float {
    if (FILL) return p.imp ? p.imp[(long long)(from + j) * c.Hkv + g] : 0.0f;
    return c.weight[row64 + j];
  };
  const bool staged = first <= stage;
  auto key_at = [&](int j) -> uint32_t { return staged ? keys[j] : order_of(weight_at(j)); };

  // the tail's weights and positions, before anything of the row is overwritten
  float tail_w = 0.0f;
  int tail_p = 0;
  if (t < tail) {
    tail_w = weight_at(body + t);
    tail_p = FILL ? body + t : c.pos[row64 + body + t];
  }

  uint32_t kth = 0;       // survivors before `first`: keys above kth,
  uint32_t ties = 0;      // and the first `ties` equal to it
  const bool all = want >= first;
  if (!all && want > 0) {
    if (staged) {
      if (FILL) {
#pragma unroll 4
        for (int j = t; j < first; j += kSelThreads) keys[j] = order_of(weight_at(j));
      } else {  // the row starts on a 256-byte boundary
        const float4* const w4 = reinterpret_cast<const float4*>(c.weight + row64);
#pragma unroll 2
        for (int j = t; j < (first + 3) / 4; j += kSelThreads) {
          const float4 v = w4[j];
          const uint32_t o[4] = {order_of(v.x), order_of(v.y), order_of(v.z), order_of(v.w)};
          if (4 * j + 3 < first) {
            *reinterpret_cast<uint4*>(keys + 4 * j) = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (4 * j + k < first) keys[4 * j + k] = o[k];
          }
        }
      }
    }
    uint32_t need = (uint32_t)want;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      hist[t] = 0;
      hist[t + kSelThreads] = 0;
      __syncthreads();
      for (int j = t; j < first; j += kSelThreads) {
        const uint32_t k = key_at(j);
        if (pass == 0 || (k >> (shift + bits)) == kth)
          atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
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
    ties = need;
  }

  // ---- ascending pass
  int32_t* const src_out = p.ws_src + (long long)row * c.cap * kTile;
  uint32_t gt_base = 0, eq_base = 0;
  const bool chosen = !all && want > 0;
  // nothing before `first` survives when want = 0
  const int begin = want > 0 ? 0 : first / kChunkTok * kChunkTok;
  for (int c0 = begin; c0 < body; c0 += kChunkTok) {
    const int j0 = c0 + 4 * t;
    bool gt[4], eq[4];
    float w[4];
    int ps[4], src[4];
    uint32_t cnt = 0;
    const int page = (!FILL && j0 < body) ? table[j0 / kTile] : 0;
    const bool bad_page = !FILL && (page < 0 || page >= c.n_pool);
    if (bad_page) atomicOr(p.status, TRA_DEV_BAD_CACHE);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + k;
      const bool in = j < body, early = j < first;
      const uint32_t key = in && early && chosen ? key_at(j) : 0u;
      gt[k] = in && (!early || all || (chosen && key > kth));
      eq[k] = in && early && chosen && key == kth;
      cnt += (gt[k] ? 0x10000u : 0u) + (eq[k] ? 1u : 0u);
      w[k] = 0.0f;
      ps[k] = j;
      src[k] = FILL ? j : (bad_page ? 0 : page) * kTile + j % kTile;
      if (gt[k] || eq[k]) {
        w[k] = early && chosen && staged ? value_of(key) : weight_at(j);
        if (!FILL) ps[k] = c.pos[row64 + j];
      }
    }
    // (a chunk holds at most 4096 of each kind: the two 16-bit halves cannot overflow)
    uint32_t sum;
    const uint32_t pre = block_scan(cnt, tmp, sum);  // its barriers: all of the chunk is read
    uint32_t gr = gt_base + (pre >> 16), er = eq_base + (pre & 0xFFFFu);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t dst = gr + min(er, ties);
      if (gt[k] || (eq[k] && er < ties)) {
        src_out[dst] = src[k];
        p.weight_out[row64 + dst] = w[k];
        p.pos_out[row64 + dst] = ps[k];
      }
      gr += gt[k];
      er += eq[k];
    }
    gt_base += sum >> 16;
    eq_base += sum & 0xFFFFu;
    __syncthreads();
  }
  if (t < tail) {
    p.weight_out[row64 + m + t] = tail_w;
    p.pos_out[row64 + m + t] = tail_p;
  }

  // ---- destination pages; an evicted row's table turns by them
  int32_t* const dst_out = p.ws_dst + (long long)row * c.cap;
  const int d0 = FILL ? 0 : body / kTile;  // first destination entry
  for (int i = t; i < n; i += kSelThreads) {
    const int page = table[d0 + i];
    const bool bad = page < 0 || page >= c.n_pool;
    if (bad) atomicOr(p.status, TRA_DEV_BAD_CACHE);
    dst_out[i] = bad ? -1 : page;
  }
  if (!FILL) {
    __syncthreads();
    const int old = d0;
    // the old pages move up by n, the last ones first
    for (int hi = old; hi > 0; hi -= kSelThreads) {
      const int i = hi - 1 - t;
      const int page = i >= 0 ? table[i] : 0;
      __syncthreads();
      if (i >= 0) table_out[n + i] = page;
      __syncthreads();
    }
    for (int i = t; i < n; i += kSelThreads) table_out[i] = dst_out[i];
    if (table_out != table)
      for (int i = old + n + t; i < c.cap; i += kSelThreads) table_out[i] = table[i];
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

// codes of fl32(s * code) for a new scale sn; ratio = s / sn
__device__ __forceinline__ uint4 recode16(uint4 v, float s, float sn, float ratio) {
  float f[16], z[16];
  floats16(v, f);
  float far = 0.0f;
  const float2 r2 = make_float2(ratio, ratio);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float2 x = make_float2(f[j], f[j + 1]);
    const float2 zz = __ffma2_rn(x, r2, make_float2(kRoundMagic, kRoundMagic));
    const float2 cn = __ffma2_rn(zz, make_float2(-1.0f, -1.0f), make_float2(kRoundMagic, kRoundMagic));
    const float2 t = __ffma2_rn(x, r2, cn);
    z[j] = zz.x;
    z[j + 1] = zz.y;
    far = fmaxf(far, fmaxf(fabsf(t.x), fabsf(t.y)));
  }
  if (far < kNearHalf && sn >= kSmallScale)
    return make_uint4(low_bytes(z[0], z[1], z[2], z[3]), low_bytes(z[4], z[5], z[6], z[7]),
                      low_bytes(z[8], z[9], z[10], z[11]), low_bytes(z[12], z[13], z[14], z[15]));
  uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    o[j >> 2] |= (uint32_t)(quant_code(__fmul_rn(s, f[j]), sn, 127) & 0xFF) << ((j & 3) * 8);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ float amax16(uint4 v) {
  float f[16];
  floats16(v, f);
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; j += 2) m = fmaxf(m, fmaxf(fabsf(f[j]), fabsf(f[j + 1])));
  return m;
}

template <int D, bool FILL>
__global__ void __launch_bounds__(256) paged_write_kernel(const PagedCutParams p) {
  __shared__ float red[16];
  const int i = blockIdx.x, g = blockIdx.y, b = blockIdx.z, t = threadIdx.x;
  const tra_paged_cache& c = p.c;
  const int4 st = p.ws_state[b];
  if (i == 0 && g == 0 && t == 0) {
    int4* const so = reinterpret_cast<int4*>(p.state_out) + b;
    int4 s = FILL ? make_int4(st.x, st.y, st.z, 0) : reinterpret_cast<const int4*>(c.state)[b];
    if (!FILL && st.w) s.x = st.x;
    *so = s;
  }
  if (!st.w) return;
  const int row = b * c.Hkv + g;
  if (FILL && i == p.keep) {  // the tail's rows
    const int from = __ldg(p.cu + b) + st.z - st.y;
    for (int f = t; f < st.y * (D / 8); f += 256) {
      const int r = f / (D / 8), ch = f % (D / 8) * 8;
      const long long src = ((long long)(from + r) * c.Hkv + g) * D + ch;
      const long long dst = ((long long)row * kTile + r) * D + ch;
      *reinterpret_cast<uint4*>(c.k_tail + dst) = *reinterpret_cast<const uint4*>(p.k + src);
      *reinterpret_cast<uint4*>(c.v_tail + dst) = *reinterpret_cast<const uint4*>(p.v + src);
    }
    return;
  }
  if (i >= st.x) return;
  const int page = p.ws_dst[(long long)row * c.cap + i];
  if (page < 0) return;
  const int32_t* const src = p.ws_src + ((long long)row * c.cap + i) * kTile;
  if constexpr (FILL) {
    const long long from = __ldg(p.cu + b);
    auto at = [&](const uint16_t* x, int r) { return x + ((from + src[r]) * c.Hkv + g) * D; };
    quantise_page<D>(c, page, [&](int r) { return at(p.k, r); }, [&](int r) { return at(p.v, r); }, red);
  } else {
    constexpr int kChunks = D / 16, kPasses = kTile * kChunks / 256;
    uint4 kx[kPasses], vx[kPasses];
    float ks[kPasses], vs[kPasses];
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      const int f = y * 256 + t;
      const int from = src[f / kChunks];
      const long long at = (long long)from * D + (f % kChunks) * 16;
      kx[y] = *reinterpret_cast<const uint4*>(c.k8 + at);
      vx[y] = *reinterpret_cast<const uint4*>(c.v8 + at);
      ks[y] = c.sk[from / kTile];
      vs[y] = c.sv[from / kTile];
    }
    // fl32(s * code) grows with |code|: the largest of a chunk is s times its largest code
    float ka = 0.0f, va = 0.0f;
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      ka = fmaxf(ka, __fmul_rn(ks[y], amax16(kx[y])));
      va = fmaxf(va, __fmul_rn(vs[y], amax16(vx[y])));
    }
    const float2 am = block_max2(ka, va, red);
    const float sk = __fdiv_rn(am.x, 127.0f), sv = __fdiv_rn(am.y, 127.0f);
    if (t == 0) {
      c.sk[page] = sk;
      c.sv[page] = sv;
    }
    int8_t* const k8 = c.k8 + (long long)page * kTile * D;
    int8_t* const v8 = c.v8 + (long long)page * kTile * D;
#pragma unroll
    for (int y = 0; y < kPasses; ++y) {
      const int f = y * 256 + t;
      *reinterpret_cast<uint4*>(k8 + f * 16) = recode16(kx[y], ks[y], sk, sk > 0.0f ? __fdiv_rn(ks[y], sk) : 0.0f);
      *reinterpret_cast<uint4*>(v8 + f * 16) = recode16(vx[y], vs[y], sv, sv > 0.0f ? __fdiv_rn(vs[y], sv) : 0.0f);
    }
  }
}

template <bool FILL>
cudaError_t launch_cut(const PagedCutParams& p, cudaStream_t s) {
  const tra_paged_cache& c = p.c;
  const int stage = p.nmax < kStageMax ? p.nmax : kStageMax;
  const size_t smem = ((size_t)stage * 4 + 15) & ~(size_t)15;
  cudaError_t e = cudaFuncSetAttribute(paged_select_kernel<FILL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMax * 4);
  if (e != cudaSuccess) return e;
  paged_select_kernel<FILL><<<dim3(c.Hkv, c.B), kSelThreads, smem, s>>>(p, stage);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid(p.keep + (FILL ? 1 : 0), c.Hkv, c.B);
  if (c.d == 128)
    paged_write_kernel<128, FILL><<<grid, 256, 0, s>>>(p);
  else
    paged_write_kernel<64, FILL><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_fill(const PagedCutParams& p, cudaStream_t s) { return launch_cut<true>(p, s); }
cudaError_t launch_paged_evict(const PagedCutParams& p, cudaStream_t s) { return launch_cut<false>(p, s); }

}  // namespace tra
