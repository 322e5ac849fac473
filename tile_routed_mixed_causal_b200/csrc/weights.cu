// weights.cu -- accumulated attention weight of a prompt's keys (the importance that
// hybrid_select_tokens and the evicting cache take): for key j and KV head g
//   w[j][g] = sum over the query heads h of g and the window's queries i >= j of
//             exp(scale q_ih . k_jg - lse[h][i]),
// and, where the caller has none, lse[h][i] = log sum_{j <= i} exp(scale q_ih . k_jg).
//
// Both are one kernel with the roles of queries and keys exchanged.  A work unit is 128
// rows (the M of one tcgen05 MMA, TMEM lanes) against a stream of 128-column tiles:
//   sums:  rows = 128 keys of one KV head, columns = queries of all heads of its group;
//          a thread owns a key and adds exp2(s c - lse2[column]), no exchange at all;
//   lse:   rows = 128 queries of one head, columns = keys; a thread owns a query and keeps
//          its running maximum and sum.
// A tile of queries holds 128 >> pack tokens of 2^pack heads of a group, token-major: one head
// in general, more where the window is short (64 queries: two heads, so the keys are read and
// multiplied for both at once).
// The scores live in TMEM and registers only.  Per element the kernel needs one product
// column of the tensor cores (d multiply-adds, 4096 per SM and cycle) and one exponential
// (16 per SM and cycle), so for d <= 128 the exponentials bound it.
// (32 heads x 32K tokens, all queries, lse given: 5.7 to 6.0 ms at the 1 kW power limit, which holds
// the SM clock at 1.72 to 1.76 GHz: 1.72e10 exponentials, 72 % of what the unit can do at that clock.
// Part of the exponentials as a polynomial on the FMA pipe: within 3 %.  Twice the softmax warps:
// 6 % slower.)
// Roles (384 threads, two CTAs per SM): warp 0 copies tiles (TMA), warp 1 issues the MMAs,
// warps 2 and 3 stage the columns' normalisers (sums only), warps 4-7 and 8-11 take the
// even and the odd tiles, one S block of TMEM each.
// Sums run in fp32: within a tile over four chains, tile sums with a compensated add, so
// that the error does not grow with the number of tiles.
// The tensor core cuts its fp32 sums off toward zero after each of the D / 16 MMAs of a score.  An lse of
// this call's own carries the same bias, and it cancels.  Over a caller's lse it would show (7e-6 of
// the sums at scores near 50), so there the accumulator starts at -f L, L = lse / scale, by one more
// MMA, of ones with the start in three bf16 parts: with f = (n + 1) / 2n of n MMAs the partial sums
// P_k - f L of a score near L are as far below zero as above it, in the mean over both orders of the
// channels (P_k + P'_(n-k) = L), which alternate from tile to tile; what is cut off, in proportion
// to the sum, cancels.  What is left for the exponential, (S - f L) - (1 - f) L, is small where a
// key has weight, so that the scale's own rounding does not show either.  Sums of 8K to 32K prompts
// are off by 2e-7 to 7e-7 (an fp32 softmax: 2e-7 to 9e-7), those of 700 tokens with scores up to 155,
// where single roundings show, by 1.2e-6 at most; the MMA costs 1 to 2 %
// of the time.
// Where there are few units a cluster of up to 8 CTAs shares one (every C-th tile each)
// and joins the partial rows over distributed shared memory in rank order: the same call
// gives the same bits.
#include "launch_ex.cuh"
#include "tra_device.cuh"
#include "tra_launch.h"

namespace tra {
namespace {

constexpr int kWThreads = 384;
constexpr int kRows = 128;   // rows of a unit, columns of a tile
constexpr int kColSlots = 4;
constexpr uint32_t kWTmemCols = 256;  // two S blocks of 128 fp32 columns
// log2 units by which a row's scores may pass its reference maximum before the sum is
// rescaled: the sum stays below 2^16 * 2^31
constexpr float kLseSlack = 16.0f;

template <int D, bool GIVEN>
struct WCfg {
  static constexpr int kTileBytes = kRows * D * 2;
  // tile ring: as deep as two CTAs per SM allow, or (lone) one
  static constexpr int kStages2 = D == 128 ? 2 : 4, kStages1 = D == 128 ? 5 : 8;
  static constexpr int kSlabs = D / 64;
  static constexpr int kOffA = 0;
  static constexpr int kOffCol = kTileBytes;                        // [kColSlots][128] float
  static constexpr int kOffFlag = kOffCol + kColSlots * kRows * 4;  // [kColSlots][2] int
  static constexpr int kOffRed = kOffFlag + kColSlots * 2 * 4;      // [2][128] float2, see red
  static constexpr int kOffBar = kOffRed + (GIVEN ? 0 : 2 * kRows * 8);
  static constexpr int kNumBars = 1 + 2 * kStages1 + 4 + 2 * kColSlots + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  // over a caller's lse: 128 rows of 16 ones, and for either S block the columns' starting values
  static constexpr int kOffX = (kOffMisc + 32 + 255) / 256 * 256;
  static constexpr int kXBytes = kRows * 32;
  // the rows' results of an S block's warps, at the end: over a caller's lse where its starting
  // values were (with another place for them two CTAs per SM have no room for four column slots, and
  // three cost 1.5 %)
  static constexpr int red(int w) { return GIVEN ? kOffX + (1 + w) * kXBytes : kOffRed + w * kRows * 8; }
  static constexpr int kOffB = (kOffX + (GIVEN ? 3 * kXBytes : 0) + 1023) / 1024 * 1024;  // the ring, last
  static constexpr int smem(int stages) { return kOffB + stages * kTileBytes + 1024; }
  // more than a third of an SM's shared memory each, so that no more than two CTAs share
  // one: their S blocks fill its TMEM
  static_assert(smem(kStages2) > 77 * 1024 && 2 * (smem(kStages2) + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(smem(kStages1) <= 227 * 1024, "one CTA per SM");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 columns of the warp's TMEM lanes, and the fence that keeps their reads behind the wait
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// this CTA's shared address `a` in CTA `rank` of the cluster
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t a, uint32_t rank) {
  uint32_t m;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(m) : "memory");
  return v;
}

__device__ __forceinline__ void mma_bf16_e(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

enum WeightPass { kPassLse, kPassSums, kPassGiven };  // kPassGiven: sums over a caller's lse

// One unit and the tiles of its stream that this CTA takes.
template <bool LSE>
struct WUnit {
  bool valid;
  int b, head;       // head: first query head of the rows (lse), KV head (sums)
  int seq0, T, wq0;  // sequence start, length, first query of the window
  int r0;            // first row's position (query or key) within the sequence
  int ncol, c0;      // column tiles per head, the first of them
  int steps;         // tiles of the stream (all CTAs of the cluster)

  // 128-row tiles of sequence i
  __device__ static __forceinline__ int tiles(const WeightParams& p, int i) {
    const int len = __ldg(p.cu + i + 1) - __ldg(p.cu + i);
    if (!LSE) return (len + kRows - 1) / kRows;
    const int W = p.n_queries > 0 ? min(len, p.n_queries) : len, qtok = kRows >> p.pack;
    return (W + qtok - 1) / qtok;
  }

  // Whole-warp call.  Units: tile t of every sequence before tile t + 1 of any, heads fastest.
  __device__ __forceinline__ void init(const WeightParams& p, long long id) {
    const int H = LSE ? p.Hq >> p.pack : p.Hkv;
    head = (int)(id % H);
    b = (int)((id / H) % p.B);
    int t = (int)(id / ((long long)H * p.B));
    if (p.ragged) {
      // very different lengths: only the tiles there are.  Tiles before t: the sum of min(tiles, t);
      // t is the largest with no more of them than this unit's index
      const int lane = threadIdx.x & 31;
      const int q = (int)(id / H);
      auto before = [&](int tt) {
        int n = 0;
        for (int i = lane; i < p.B; i += 32) n += min(tiles(p, i), tt);
        return __reduce_add_sync(0xffffffffu, n);
      };
      int lo = 0, hi = LSE ? p.lse_tiles : p.sum_tiles;  // before(lo) <= q < before(hi)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before(mid) <= q) lo = mid;
        else hi = mid;
      }
      t = lo;
      int r = q - before(t);  // the r-th sequence that has a tile t
      for (int i0 = 0; i0 < p.B; i0 += 32) {
        const uint32_t has = __ballot_sync(0xffffffffu, i0 + lane < p.B && tiles(p, i0 + lane) > t);
        const int n = __popc(has);
        if (r < n) {
          b = i0 + (int)__fns(has, 0, r + 1);
          break;
        }
        r -= n;
      }
    }
    seq0 = __ldg(p.cu + b);
    T = __ldg(p.cu + b + 1) - seq0;
    const int W = p.n_queries > 0 ? min(T, p.n_queries) : T;
    const int qtok = kRows >> p.pack;  // tokens of a query tile
    const int nq = (W + qtok - 1) / qtok;
    wq0 = T - W;
    if (LSE) {  // query tiles count from the window's first query; the longest rows first
      head <<= p.pack;
      valid = t < nq;
      r0 = wq0 + (nq - 1 - t) * qtok;
      c0 = 0;
      ncol = valid ? (min(r0 + qtok, T) - 1) / kRows + 1 : 0;  // key tiles 0 .. that of the last row
      steps = ncol;
    } else {  // key tiles in order: the first are seen by the most queries
      valid = t * kRows < T;
      r0 = t * kRows;
      c0 = r0 > wq0 ? (r0 - wq0) / qtok : 0;  // earlier tiles end before the first key
      ncol = nq - c0;
      steps = valid ? ncol * ((p.Hq / p.Hkv) >> p.pack) : 0;
    }
  }
  // step u: (first) query head and first query (sums), or first key (lse) of the column tile
  __device__ __forceinline__ void column(const WeightParams& p, int u, int& h, int& x0) const {
    if (LSE) {
      h = head / (p.Hq / p.Hkv);
      x0 = u * kRows;
    } else {
      h = head * (p.Hq / p.Hkv) + (u / ncol << p.pack);
      x0 = wq0 + (c0 + u % ncol) * (kRows >> p.pack);
    }
  }
};

template <int D, WeightPass PASS>
__global__ void __launch_bounds__(kWThreads, 2)
    weight_kernel(const __grid_constant__ WeightParams p, const __grid_constant__ WeightMaps m) {
  constexpr bool LSE = PASS == kPassLse, GIVEN = PASS == kPassGiven;
  using C = WCfg<D, GIVEN>;
  extern __shared__ uint8_t wsm_raw[];
  const uint32_t base = (smem_u32(wsm_raw) + 1023u) & ~1023u;
  uint8_t* const gbase = wsm_raw + (base - smem_u32(wsm_raw));
  const uint32_t rank = cluster_rank(), nrank = cluster_size();
  if (LSE) grid_release();
  WUnit<LSE> x;
  x.init(p, blockIdx.x / nrank);
  if (!x.valid) return;  // the whole cluster leaves
  const int nsteps = (x.steps - (int)rank + (int)nrank - 1) / (int)nrank;  // this CTA's, may be 0

  const uint32_t bars = base + C::kOffBar;
  const uint32_t bar_a = bars;
  auto bar_bfull = [&](int s) { return bars + (1 + s) * 8; };
  auto bar_bfree = [&](int s) { return bars + (1 + C::kStages1 + s) * 8; };
  constexpr int kSB = 1 + 2 * C::kStages1;
  const int stages = p.stages;
  auto bar_sfull = [&](int w) { return bars + (kSB + w) * 8; };
  auto bar_sfree = [&](int w) { return bars + (kSB + 2 + w) * 8; };
  auto bar_cfull = [&](int s) { return bars + (kSB + 4 + s) * 8; };
  auto bar_cfree = [&](int s) { return bars + (kSB + 4 + kColSlots + s) * 8; };
  const uint32_t bar_done = bars + (kSB + 4 + 2 * kColSlots) * 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int* const err = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 16);
  float* const col = reinterpret_cast<float*>(gbase + C::kOffCol);
  volatile int* const flag = reinterpret_cast<volatile int*>(gbase + C::kOffFlag);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    prefetch_map(&m.q);
    prefetch_map(&m.k);
  }
  if (threadIdx.x == 0) {
    mbar_init(bar_a, 1);
    for (int s = 0; s < stages; ++s) {
      mbar_init(bar_bfull(s), 1);
      mbar_init(bar_bfree(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar_sfull(w), 1);
      mbar_init(bar_sfree(w), 4);
    }
    for (int s = 0; s < kColSlots; ++s) {
      mbar_init(bar_cfull(s), 64);
      mbar_init(bar_cfree(s), 4);
    }
    mbar_init(bar_done, 1);
    *err = 0;
    fence_barrier_init();
  }
  if constexpr (GIVEN) {  // bf16 ones in every place of the rows' 32 bytes, zeroes in the columns'
    for (int i = threadIdx.x; i < 3 * C::kXBytes / 16; i += kWThreads) {
      const uint32_t v = i < C::kXBytes / 16 ? 0x3F803F80u : 0u;
      reinterpret_cast<uint4*>(gbase + C::kOffX)[i] = make_uint4(v, v, v, v);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kWTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wwait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
  };

  // a row's result: sums (total, -), lse (reference maximum, sum)
  float2 part = make_float2(LSE ? -INFINITY : 0.0f, 0.0f);

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    const CUtensorMap* const ma = LSE ? &m.q : &m.k;
    const CUtensorMap* const mb = LSE ? &m.k : &m.q;
    mbar_arrive_expect_tx_e(bar_a, C::kTileBytes);
    for (int sl = 0; sl < C::kSlabs; ++sl)
      tma_load_3d_e(base + C::kOffA + sl * kRows * 128, ma, bar_a, sl * 64, x.head, x.seq0 + x.r0);
    int n = 0;
    for (; n < nsteps; ++n) {
      const int s = n % stages, use = n / stages;
      if (use > 0 && !wwait(bar_bfree(s), (use - 1) & 1)) break;
      int h, x0;
      x.column(p, (int)rank + n * (int)nrank, h, x0);
      mbar_arrive_expect_tx_e(bar_bfull(s), C::kTileBytes);
      for (int sl = 0; sl < C::kSlabs; ++sl)
        tma_load_3d_e(base + C::kOffB + s * C::kTileBytes + sl * kRows * 128, mb, bar_bfull(s), sl * 64, h,
                      x.seq0 + x0);
    }
    // every copy lands before the CTA can leave (only this warp arrives on these barriers)
    if (nsteps == 0 || *err) {
      mbar_wait_drain(bar_a, 0);
      for (int s = 0; s < stages && s < n; ++s)
        mbar_wait_drain(bar_bfull(s), (uint32_t)(((n - 1 - s) / stages) & 1));
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t kId = instr_desc(1, 1, 0, 0, kRows, 128);
    const uint64_t dA = smem_desc(base + C::kOffA, 16, 1024, kSwz128);
    bool ok = nsteps > 0 && wwait(bar_a, 0);
    for (int n = 0; ok && n < nsteps; ++n) {
      const int s = n % stages, w = n & 1;
      // S block w last held tile n - 2; its warps have read it into registers
      if (n >= 2 && !wwait(bar_sfree(w), ((n >> 1) - 1) & 1)) break;
      if (!wwait(bar_bfull(s), (n / stages) & 1)) break;
      if (GIVEN && !wwait(bar_cfull(n % kColSlots), (n / kColSlots) & 1)) break;
      tc_fence_after();
      if (GIVEN)  // the starting values
        mma_bf16_e(tmem + w * kRows, smem_desc(base + C::kOffX, 16, 256, kSwz32),
                   smem_desc(base + C::kOffX + (1 + w) * C::kXBytes, 16, 256, kSwz32), kId, 0u);
      const uint64_t dB = smem_desc(base + C::kOffB + s * C::kTileBytes, 16, 1024, kSwz128);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {  // 16 channels: 32 bytes within a 64-channel slab of 16 KB
        const int kk = GIVEN && (n & 1) ? D / 16 - 1 - i : i;
        const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;
        mma_bf16_e(tmem + w * kRows, dA + off, dB + off, kId, GIVEN || i > 0 ? 1u : 0u);
      }
      mma_commit_e(bar_bfree(s));
      mma_commit_e(bar_sfull(w));
    }
    // every MMA is complete before TMEM is released
    mma_commit_e(bar_done);
    mbar_wait_drain(bar_done, 0);
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- column normalisers
    if (!LSE) {
      grid_wait();  // the lse may be the preceding launch's
      const int c = (warp - 2) * 64 + lane;  // and c + 32
      for (int n = 0; n < nsteps; ++n) {
        const int s = n % kColSlots, use = n / kColSlots;
        int h, x0;
        x.column(p, (int)rank + n * (int)nrank, h, x0);
        const float* const src = p.lse + (long long)h * p.ntok + x.seq0;
        float z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = x0 + ((c + 32 * k) >> p.pack);
          z[k] = i < x.T ? src[((c + 32 * k) & ((1 << p.pack) - 1)) * p.ntok + i] : INFINITY;
        }
        if (use > 0 && !wwait(bar_cfree(s), (use - 1) & 1)) break;
        // the starting values' tile was last read by the MMAs of tile n - 2
        if (GIVEN && n >= 2 && !wwait(bar_sfull(n & 1), ((n >> 1) - 1) & 1)) break;
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const bool fin = isfinite(z[k]);  // a row that is not finite adds nothing
          odd |= !fin;
          float v = z[k] * -1.4426950408889634f;
          if constexpr (GIVEN) {
            constexpr int kMmas = D / 16;
            const double L = fin ? (double)z[k] * p.inv_scale : 0.0;
            // (beyond 2^60 every exponential is zero or infinite)
            const float a = fminf(fmaxf((float)(L * (-0.5 * (kMmas + 1) / kMmas)), -0x1p60f), 0x1p60f);
            v = (float)((-(double)a - L) * (double)p.scale_log2);
            // a in three bf16 parts, exactly
            const __nv_bfloat16 hi = __float2bfloat16_rn(a);
            const float r = a - __bfloat162float(hi);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(r, r - __bfloat162float(__float2bfloat16_rn(r)));
            *reinterpret_cast<uint2*>(gbase + C::kOffX + (1 + (n & 1)) * C::kXBytes + (c + 32 * k) * 32) =
                make_uint2(*reinterpret_cast<const uint16_t*>(&hi), *reinterpret_cast<const uint32_t*>(&lo));
          }
          col[s * kRows + c + 32 * k] = fin ? v : -INFINITY;
        }
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) flag[s * 2 + warp - 2] = odd;
        if (GIVEN) fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive(bar_cfull(s));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax warps
    const int w = (warp - 4) >> 2;                    // tile parity, S block
    const int r = (warp & 3) * 32 + lane;             // row = TMEM lane
    const int row = x.r0 + (LSE ? r >> p.pack : r);   // query or key position
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(w * kRows);
    const float c1 = p.scale_log2;
    const float2 c2 = make_float2(c1, c1);
    const bool warp_rows = x.r0 + ((warp & 3) * 32 >> (LSE ? p.pack : 0)) < x.T;
    float total = 0.0f, comp = 0.0f;                  // sums: compensated total
    float mref = -INFINITY, l = 0.0f;                 // lse
    for (int n = w; n < nsteps; n += 2) {
      const int cs = n % kColSlots;
      int h, x0;
      x.column(p, (int)rank + n * (int)nrank, h, x0);
      if (!LSE && !mbar_wait(bar_cfull(cs), (n / kColSlots) & 1, err)) break;
      if (!mbar_wait(bar_sfull(w), (n >> 1) & 1, err)) break;
      __syncwarp();
      tc_fence_after();
      // the S block is free for the tile after next once its last columns are in registers
      auto release_s = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sfree(w));
      };
      // a full tile: 16 columns at a time, unrolled, the next 16 on their way meanwhile
      auto pipelined = [&](auto body) {
        uint32_t ra[16], rb[16];
        tmem_ld16(tS, ra);
#pragma unroll
        for (int c0 = 0; c0 < kRows; c0 += 32) {
          tmem_wait_ld();
          reg_fence16(ra);
          tmem_ld16(tS + c0 + 16, rb);
          body(c0, ra);
          tmem_wait_ld();
          reg_fence16(rb);
          if (c0 + 32 < kRows) tmem_ld16(tS + c0 + 32, ra);
          else release_s();
          body(c0 + 16, rb);
        }
      };
      if (!warp_rows) {  // no row of this warp exists: the tile only passes through
        release_s();
      } else if (LSE) {
        // keys behind the last row of the sequence are behind every valid row, too
        const bool masked = x0 + kRows - 1 > x.r0;
        const int nchunk = min(kRows, x.T - x0 + 31) >> 5;
        auto add = [&](auto& sr) {  // these columns into the row's maximum and sum
          constexpr int N = sizeof(sr) / 4;
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = __uint_as_float(sr[k]);
#pragma unroll
          for (int k = 4; k < N; ++k) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(sr[k]));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1;
          if (mt > mref + kLseSlack || (mref == -INFINITY && mt > mref)) {
            l *= ex2(mref - mt);  // mref = -inf gives 0
            mref = mt;
          }
          const float nm = mref == -INFINITY ? 0.0f : -mref;
          float2 a[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int k = 0; k < N; k += 2) {
            const float2 e = __ffma2_rn(make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), c2, make_float2(nm, nm));
            a[(k >> 1) & 1] = __fadd2_rn(a[(k >> 1) & 1], make_float2(ex2(e.x), ex2(e.y)));
          }
          const float2 s2 = __fadd2_rn(a[0], a[1]);
          l += s2.x + s2.y;
        };
        if (!masked && nchunk == 4) {
          pipelined([&](int, uint32_t (&sr)[16]) { add(sr); });
        } else {
#pragma unroll 1
          for (int ch = 0; ch < nchunk; ++ch) {
            uint32_t sr[32];
            tmem_ld32(tS + 32 * ch, sr);
            tmem_wait_ld();
            tmem_reg_fence(sr);
            if (ch == nchunk - 1) release_s();
            const int lim = row - (x0 + 32 * ch);  // columns 0 .. lim are visible
#pragma unroll
            for (int k = 0; k < 32; ++k) sr[k] = k <= lim ? sr[k] : 0xFF800000u;
            add(sr);
          }
        }
      } else {
        // queries before the key, past the window's end or without a finite lse add
        // nothing; where a tile has such columns they are selected away one by one, since
        // a score there may be anything
        const bool masked = x0 < x.r0 + kRows - 1 || flag[cs * 2] || flag[cs * 2 + 1];
        const int nchunk = (min(kRows, (x.T - x0) << p.pack) + 31) >> 5;
        const float4* const nl = reinterpret_cast<const float4*>(col + cs * kRows);
        float2 a[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        if (!masked && nchunk == 4) {
          pipelined([&](int c0, uint32_t (&sr)[16]) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 z = nl[(c0 + k) / 4];
              const float2 s0 = make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1]));
              const float2 s1 = make_float2(__uint_as_float(sr[k + 2]), __uint_as_float(sr[k + 3]));
              const float2 e0 = __ffma2_rn(s0, c2, make_float2(z.x, z.y)), e1 = __ffma2_rn(s1, c2, make_float2(z.z, z.w));
              a[0] = __fadd2_rn(a[0], make_float2(ex2(e0.x), ex2(e0.y)));
              a[1] = __fadd2_rn(a[1], make_float2(ex2(e1.x), ex2(e1.y)));
            }
          });
        } else {
#pragma unroll 1
          for (int ch = 0; ch < nchunk; ++ch) {
            uint32_t sr[32];
            tmem_ld32(tS + 32 * ch, sr);
            tmem_wait_ld();
            tmem_reg_fence(sr);
            if (ch == nchunk - 1) release_s();
            const int lim = ((row - x0) << p.pack) - 32 * ch;  // columns from lim on see the key
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 z = nl[8 * ch + k / 4];
              const float zz[4] = {z.x, z.y, z.z, z.w};
              float e[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                e[y] = ex2(fmaf(__uint_as_float(sr[k + y]), c1, zz[y]));
                if (k + y < lim || zz[y] == -INFINITY) e[y] = 0.0f;
              }
              a[0] = __fadd2_rn(a[0], make_float2(e[0], e[1]));
              a[1] = __fadd2_rn(a[1], make_float2(e[2], e[3]));
            }
          }
        }
        const float2 s2 = __fadd2_rn(a[0], a[1]);
        // compensated add: comp carries what the total could not hold
        const float y = __fsub_rn(s2.x + s2.y, comp);
        const float t = __fadd_rn(total, y);
        comp = t < INFINITY ? __fsub_rn(__fsub_rn(t, total), y) : 0.0f;  // (an infinite sum stays one)
        total = t;
      }
      if (!LSE) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_cfree(cs));
      }
    }
    part = LSE ? make_float2(mref, l) : make_float2(total, 0.0f);
    reinterpret_cast<float2*>(gbase + C::red(w))[r] = part;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kWTmemCols);  // before the wait for other CTAs
  if (threadIdx.x == 0 && *err) atomicOr(p.status, *err);

  // join the CTAs' rows, even tiles then odd ones of each rank
  if (nrank > 1) cluster_sync();
  const int row = x.r0 + (LSE ? (int)threadIdx.x >> p.pack : (int)threadIdx.x);
  if (rank == 0 && threadIdx.x < kRows && row < x.T) {
    const uint32_t red = base + threadIdx.x * 8;
    float mm = -INFINITY, acc = 0.0f;
    if (LSE)
      for (uint32_t k = 0; k < nrank; ++k)
        for (int w = 0; w < 2; ++w) mm = fmaxf(mm, ld_cluster_f2(red + C::red(w), k).x);
    for (uint32_t k = 0; k < nrank; ++k)
      for (int w = 0; w < 2; ++w) {
        const float2 v = ld_cluster_f2(red + C::red(w), k);
        if (LSE) acc += v.x == -INFINITY ? 0.0f : v.y * ex2(v.x - mm);
        else acc += v.x;
      }
    if (LSE)
      p.lse[(long long)(x.head + (threadIdx.x & ((1 << p.pack) - 1))) * p.ntok + x.seq0 + row] = (mm + log2f(acc)) * 0.69314718055994531f;
    else
      p.weights[(long long)(x.seq0 + row) * p.Hkv + x.head] = acc;
  }
  __syncwarp();
  if (nrank > 1) cluster_sync();  // a CTA's rows stay until rank 0 has read them
}

template <int D, WeightPass PASS>
cudaError_t launch_weight_pass(WeightParams p, const WeightMaps& m, bool overlap, cudaStream_t s) {
  using C = WCfg<D, PASS == kPassGiven>;
  constexpr bool LSE = PASS == kPassLse;
  const long long units = LSE ? p.lse_units : p.sum_units, longest = LSE ? p.lse_longest : p.sum_longest;
  // CTAs per unit: as few as bring the longest unit near the mean load of the grid's 296
  // places (two per SM), so that a short stream of units still fills the GPU
  const long long steps = LSE ? p.lse_steps : p.sum_steps, mean = steps / 296 > 4 ? steps / 296 : 4;
  int cluster = 1;
  while (cluster < 8 && (longest + cluster - 1) / cluster > mean) cluster *= 2;
  const long long ctas = units * cluster;
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  // a grid of at most one CTA per SM has each alone: the deeper ring.  (Only 15 clusters of 8
  // such CTAs fit the GPU at a time: a 16th, as a second wave, would double the time.)
  p.stages = ctas <= 120 ? C::kStages1 : C::kStages2;
  static SmemLimit limit;
  cudaError_t e = limit.raise(weight_kernel<D, PASS>, C::smem(C::kStages1));
  if (e != cudaSuccess) return e;
  return launch_ex(weight_kernel<D, PASS>, dim3((unsigned)ctas), kWThreads, C::smem(p.stages), s, cluster, overlap, p, m);
}

template <int D>
cudaError_t launch_weight_d(const WeightParams& p, const WeightMaps& m, cudaStream_t s) {
  if (p.lse_given) return launch_weight_pass<D, kPassGiven>(p, m, false, s);
  cudaError_t e = launch_weight_pass<D, kPassLse>(p, m, false, s);
  return e != cudaSuccess ? e : launch_weight_pass<D, kPassSums>(p, m, true, s);
}

}  // namespace

cudaError_t launch_weight_sums(const WeightParams& p, const WeightMaps& m, cudaStream_t s) {
  return p.d == 128 ? launch_weight_d<128>(p, m, s) : launch_weight_d<64>(p, m, s);
}

}  // namespace tra
