// paged_decode.cu -- one decode step over the evicting cache: attention over a row's INT8
// pages, its bf16 tail and the new token, the probabilities added to the tokens' weights,
// and the append.
//
// Attention.  The pages of all rows (a row = one sequence and KV head) and one tail item per
// row form one list, which the grid's CTAs (two per SM) share in equal contiguous pieces:
// ragged rows and single long ones load every SM alike.  A CTA is a producer warp and four
// consumer warps.  The producer streams pages (8 KB of K codes, 8 KB of V codes at d = 128,
// TMA with the swizzle that makes the reads below bank-conflict free) through a ring; each
// consumer warp takes every fourth page (a quarter of every page, where there are few) with its
// own softmax state for all query heads of the group, so every cached byte is read once:
//   S = K q:    mma m16n8k16, M = 16 keys, N = 8 heads.  K codes become f16 exactly; q is
//               scaled per head by a power of two so that its bf16 values are f16 exactly
//               (all within 2^31 of the head's largest), products are exact and summed in fp32:
//               the scores that the weights are made of lose nothing to quantised queries;
//   softmax:    lazily rescaled running maximum and sum in fp32, log2 domain;
//   O += P V:   p as a pair of f16, hi + lo (22 bits: f16 alone showed where values cancel), transposed
//               between the fragments by movmatrix, each with a chain of MMAs of its own (in one
//               chain: 3 % slower on a ragged batch; the pair itself costs 0 to 1 %); the page's
//               V scale is applied to the fp32 product, so no small scale is lost in f16.
// A tail item (up to 64 bf16 rows) is split over the four warps, 16 rows each, straight from
// global memory with bf16 MMAs; its P goes in as a bf16 pair hi + lo.
// Every score is written once (fp32, log2 domain) and each piece leaves (m, l, O).
//
// Finish.  A second kernel, over chunks of each row's tokens, joins the row's pieces in order,
// turns the scores into probabilities with the row's m and l, adds them to the weights, writes
// the output and the new state, and quantises a tail that became full.  The split is what
// bounds the step: 2 d bytes of codes per cached token, against 4 grp + 8 bytes here.
// On the GPU, batch 16 x 32K, 32/8 heads, d 128: split 176 us (6.2 TB/s, 95 % of a copy), step 208 us;
// a single row of 2K tokens: 9.6 us.
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "launch_ex.cuh"
#include "paged_device.cuh"

namespace tra {
namespace {

constexpr int kCons = 4;                       // consumer warps
constexpr int kStepThreads = 32 * (kCons + 1);
constexpr int kPieces = 296;                   // CTAs of the list: two per SM
constexpr int kFinThreads = 128;
constexpr int kSplitItems = 8;                 // items of a piece up to which its pages are split
constexpr float kSlack = 8.0f;                 // log2 units p may pass 1 before a rescale

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit values across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// TMA copy of a page, which nobody reads again in this step: first to leave the L2 cache, so
// that the scores stay there for the finish
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t y, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(y), "l"(pol)
      : "memory");
}
// two bytes of x (biased by 128) as exact f16
__device__ __forceinline__ uint32_t h2_of(uint32_t x, uint32_t sel) {
  uint32_t h = __byte_perm(x, 0x6464u, sel);  // 1024 + byte
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(0x64806480u));
  return h;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ uint32_t pack_b2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Byte offset of 16-byte chunk c of row r in a page whose rows are R bytes, as TMA writes
// it with an R-byte swizzle.
template <int R>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  return r * R + ((c ^ ((r * R >> 7) & (R / 16 - 1))) << 4);
}
__device__ __forceinline__ void cons_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kCons) : "memory"); }

// Items (pages and the tail) that row state `st` adds per KV head; 0: the row takes no part.
__device__ __forceinline__ int row_items(int4 st, int cap) {
  if (paged_row(st, cap) != kRowOk || (st.y == kTile - 1 && st.x == cap)) return 0;
  return st.x + 1;
}

// The list: rows b-major, KV head within, a row's pages then its tail.  (Whole-warp calls.)
struct ListPos {
  int b, g, item;
};
// A list of fewer items than this is shared out in 32-bit arithmetic: the 64-bit divisions were a
// tenth of a short step.
constexpr long long kShortList = 1ll << 22;
// pieces in use, and the first item of piece i
__device__ __forceinline__ int pieces_of(long long items) { return items < kPieces ? (int)items : kPieces; }
__device__ __forceinline__ long long piece_start(long long items, int pieces, int i) {
  if (items < kShortList) return (uint32_t)items * (uint32_t)i / (uint32_t)pieces;
  return items * i / pieces;
}

// Items before this lane's sequence b0 + lane (lo) and behind it (hi), `base` before the chunk.
__device__ __forceinline__ void list_chunk(int items, int Hkv, long long base, long long& lo, long long& hi) {
  const int lane = threadIdx.x & 31;
  long long s = (long long)items * Hkv;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  hi = base + s;
  lo = hi - (long long)items * Hkv;
}

// Piece `piece` of the list: its first item and the one behind its last; pos: the sequence,
// KV head and item within the row of the first.  False: no such piece.
__device__ __forceinline__ bool list_piece(const int4* state, int B, int Hkv, int cap, int piece, long long& first,
                                           long long& last, ListPos& pos) {
  const int lane = threadIdx.x & 31;
  const int it0 = lane < B ? row_items(state[lane], cap) : 0;  // the first 32 sequences
  long long lo0, hi0;
  list_chunk(it0, Hkv, 0, lo0, hi0);
  const long long base1 = __shfl_sync(0xffffffffu, hi0, 31);
  long long items = base1;
  for (int b0 = 32; b0 < B; b0 += 32) {
    const long long n = b0 + lane < B ? (long long)row_items(state[b0 + lane], cap) * Hkv : 0;
    long long s = n;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    items += s;
  }
  const int pieces = pieces_of(items);
  if (piece >= pieces) return false;
  first = piece_start(items, pieces, piece);
  last = piece_start(items, pieces, piece + 1);
  int it = it0, b0 = 0;
  long long lo = lo0, hi = hi0;
  while (true) {  // the chunk of sequences that holds it (there is one)
    const uint32_t hit = __ballot_sync(0xffffffffu, hi > lo && first >= lo && first < hi);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const long long at = first - __shfl_sync(0xffffffffu, lo, src);
      const int n = __shfl_sync(0xffffffffu, it, src);
      pos.b = b0 + src;
      if (items < kShortList) {
        pos.g = (int)((uint32_t)at / (uint32_t)n);
        pos.item = (int)((uint32_t)at % (uint32_t)n);
      } else {
        pos.g = (int)(at / n);
        pos.item = (int)(at % n);
      }
      return true;
    }
    const long long base = __shfl_sync(0xffffffffu, hi, 31);
    b0 += 32;
    if (b0 >= B) return false;
    it = b0 + lane < B ? row_items(state[b0 + lane], cap) : 0;
    list_chunk(it, Hkv, base, lo, hi);
  }
}

template <int D, int GRP>
struct StepCfg {
  static constexpr int kTileBytes = kTile * D;       // codes of a page of K (or V)
  static constexpr int kStageBytes = 2 * kTileBytes;
  // as many stages as two CTAs per SM leave room for, at most 8
  static constexpr int kRedBytes = kCons * GRP * (D + 2) * 4;
  static constexpr int kRoom = 112 * 1024 - 1024 - kRedBytes - 512;
  static constexpr int kFit = kRoom / kStageBytes;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static_assert(kStages >= kCons, "the consumers' parity waits need a stage per warp");
  static constexpr int kOffRed = kStages * kStageBytes;
  static constexpr int kOffScale = kOffRed + kRedBytes;  // [stage] float2 (sK, sV)
  static constexpr int kOffBar = kOffScale + kStages * 8;
  static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
};

// SPLIT: the warps share every page, 16 keys each (pieces are short: a page's own latency is what the
// step waits for).
template <int D, int GRP, bool SPLIT>
__global__ void __launch_bounds__(kStepThreads, 2)
    paged_step_kernel(const __grid_constant__ PagedStepParams p, const __grid_constant__ PagedMaps m) {
  using C = StepCfg<D, GRP>;
  constexpr int kBlk = D / 16;  // 16-channel blocks
  extern __shared__ uint8_t psm_raw[];
  const uint32_t base = (smem_u32(psm_raw) + 1023u) & ~1023u;
  uint8_t* const sm = psm_raw + (base - smem_u32(psm_raw));
  float* const red = reinterpret_cast<float*>(sm + C::kOffRed);
  float2* const scale = reinterpret_cast<float2*>(sm + C::kOffScale);
  const uint32_t bar_full = base + C::kOffBar, bar_empty = bar_full + C::kStages * 8;
  volatile int* const err = reinterpret_cast<volatile int*>(sm + C::kOffMisc);
  const tra_paged_cache& c = p.c;
  const int4* const state = reinterpret_cast<const int4*>(c.state);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int grp = c.Hq / c.Hkv;

  grid_release();
  if (t == 32 * kCons) {
    prefetch_map(&m.k8);
    prefetch_map(&m.v8);
  }
  if (t == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + s * 8, 2);  // the copies' bytes, and the scales
      mbar_init(bar_empty + s * 8, SPLIT ? kCons : 1);
    }
    *err = 0;
    fence_barrier_init();
  }
  // the states as this step finds them, for the finish (which may write them in place)
  if (blockIdx.x == 0)
    for (int b = t; b < c.B; b += kStepThreads) p.ws_state[b] = state[b];
  ListPos pos{0, 0, 0};
  long long lo = 0, hi = 0;
  if (!list_piece(state, c.B, c.Hkv, c.cap, blockIdx.x, lo, hi, pos)) return;  // uniform
  __syncthreads();

  // the piece row by row: row state st, items [i0, i1) of it, the row's last item its tail
  auto for_rows = [&](auto body) {
    int b = pos.b, g = pos.g, i0 = pos.item;
    long long left = hi - lo;
    int4 st = state[b];
    while (left > 0) {
      const int n = st.x + 1;
      const int i1 = (int)min((long long)n, i0 + left);
      if (!body(b, g, st, i0, i1)) break;
      left -= i1 - i0;
      i0 = 0;
      if (left > 0 && ++g == c.Hkv) {
        g = 0;
        do st = state[++b]; while (row_items(st, c.cap) == 0);  // items are left: a row follows
      }
    }
  };

  if (warp == kCons) {
    // ---------------------------------------------------------------- producer
    int issued = 0, scaled = 0, first = 0;  // pages copied, pages with scales, first of the batch
    bool any_bad = false;
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    for_rows([&](int b, int g, int4 st, int i0, int i1) -> bool {
      const int32_t* const tab = c.table + ((long long)b * c.Hkv + g) * c.cap;
      const int end = min(i1, st.x);
      // a head whose page numbers are not all in order, that of a full tail's page among them, gives
      // nothing (paged_finish_kernel): what page 0 stands in for is another row's
      bool bad = false;
      const int next_page = i1 == st.x + 1 && st.y == kTile - 1 ? tab[st.x] : 0;  // (looked at last)
      // page numbers and scales 32 at a time, a batch ahead
      int page = 0;
      float2 sc = make_float2(0.0f, 0.0f);
      auto fetch = [&](int i) {
        page = i + lane < end ? tab[i + lane] : 0;
        if (page < 0 || page >= c.n_pool) {
          bad = true;
          page = 0;
        }
        sc = make_float2(__ldg(c.sk + page), __ldg(c.sv + page));
      };
      if (i0 < end) fetch(i0);
      for (int i = i0; i < end; i += 32) {
        const int pg = page;
        const float2 sg = sc;
        if (i + 32 < end) fetch(i + 32);
        const int cnt = min(32, end - i);
        // the first stages' copies start on the page numbers alone; their scales, another load
        // later, follow together, and from then on each page's with its copy
        for (int k = 0; k < cnt; ++k, ++issued) {
          const int s = issued % C::kStages, use = issued / C::kStages;
          if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(bar_empty + s * 8, (use - 1) & 1, err))) return false;
          const int pk = __shfl_sync(0xffffffffu, pg, k);
          if (lane == 0) {
            const uint32_t dst = base + s * C::kStageBytes;
            mbar_arrive_expect_tx(bar_full + s * 8, C::kStageBytes);
            tma_load_page(dst, &m.k8, bar_full + s * 8, pk * kTile, pol);
            tma_load_page(dst + C::kTileBytes, &m.v8, bar_full + s * 8, pk * kTile, pol);
          }
          if (issued < C::kStages - 1 && k < cnt - 1) continue;
          for (; scaled - first <= k; ++scaled) {
            const float sx = __shfl_sync(0xffffffffu, sg.x, scaled - first), sy = __shfl_sync(0xffffffffu, sg.y, scaled - first);
            if (lane == 0) {
              scale[scaled % C::kStages] = make_float2(sx, sy);
              mbar_arrive(bar_full + scaled % C::kStages * 8);
            }
          }
        }
        first = scaled;
      }
      bad = __any_sync(0xffffffffu, bad || next_page < 0 || next_page >= c.n_pool);
      if (lane == 0) {
        int32_t* const slot = p.bad + blockIdx.x + b * c.Hkv + g;
        slot[0] = bad;
        // the next row's, or, where the piece ends with the row, nobody's: a sequence is read as a whole
        if (i1 == st.x + 1) slot[1] = 0;
      }
      any_bad |= bad;
      return true;
    });
    if (any_bad && lane == 0) atomicOr(p.status, TRA_DEV_BAD_CACHE);
    // an abandoned piece: every copy lands before the CTA leaves
    if (*err) {
      for (; scaled < issued; ++scaled)
        if (lane == 0) mbar_arrive(bar_full + scaled % C::kStages * 8);
      for (int s = 0; s < C::kStages && s < issued; ++s)
        mbar_wait_drain(bar_full + s * 8, (uint32_t)(((issued - 1 - s) / C::kStages) & 1));
    }
  } else {
    // ---------------------------------------------------------------- consumers
    const int g4 = lane >> 2, tq = lane & 3;
    const int mrow = (lane & 7) + 8 * ((lane >> 3) & 1), mch = lane >> 4;  // ldmatrix row, chunk
    const int gs = paged_score_stride(grp);
    int next = SPLIT ? 0 : warp;  // this warp's next page in the piece's stream of pages
    int seen = 0;     // pages of the rows before
    bool ok = true;   // once a wait has run out: no more pages, but every barrier
    for_rows([&](int b, int g, int4 st, int i0, int i1) -> bool {
      const int row = b * c.Hkv + g;
      const long long hq = (long long)b * c.Hq + g * grp;  // first query head
      const int end = min(i1, st.x), npage = max(0, end - i0);
      float* const srow = p.scores + (long long)row * (c.cap + 1) * kTile * gs;
      // q of head g4: channels 16 j + 4 tq .. + 3
      uint2 qb[kBlk];
#pragma unroll
      for (int j = 0; j < kBlk; ++j)
        qb[j] = g4 < grp ? __ldg(reinterpret_cast<const uint2*>(p.q + (hq + g4) * D + 16 * j + 4 * tq)) : make_uint2(0, 0);
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < kBlk; ++j)
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(__uint_as_float(qb[j].x << 16)), fabsf(__uint_as_float(qb[j].x & 0xFFFF0000u))),
                             fmaxf(fabsf(__uint_as_float(qb[j].y << 16)), fabsf(__uint_as_float(qb[j].y & 0xFFFF0000u)))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int e = 0;
      frexpf(mx, &e);  // |q| < 2^e
      e = max(e, -100);  // the factors below stay finite
      const float up = ldexpf(1.0f, 15 - e);
      uint2 qh[kBlk];
#pragma unroll
      for (int j = 0; j < kBlk; ++j) {
        qh[j].x = pack_h2(__uint_as_float(qb[j].x << 16) * up, __uint_as_float(qb[j].x & 0xFFFF0000u) * up);
        qh[j].y = pack_h2(__uint_as_float(qb[j].y << 16) * up, __uint_as_float(qb[j].y & 0xFFFF0000u) * up);
      }
      // this lane's columns of S: heads 2 tq and 2 tq + 1
      const float down = ldexpf(p.scale_log2, e - 15);
      float hs[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) hs[h] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + h));

      float mr[2] = {-INFINITY, -INFINITY}, lr[2] = {0.0f, 0.0f};
      float o[kBlk][4];
#pragma unroll
      for (int j = 0; j < kBlk; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[j][k] = 0.0f;

      // running maximum of both heads to cover mt (per head over the warp); O and l follow
      auto raise = [&](const float (&mt)[2]) {
        const bool need = mt[0] > mr[0] + kSlack || mt[1] > mr[1] + kSlack;  // true from -inf
        if (!__any_sync(0xffffffffu, need)) return;
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(mr[h], mt[h]);
          al[h] = mn == -INFINITY ? 1.0f : ex2(mr[h] - mn);
          mr[h] = mn;
          lr[h] *= al[h];
        }
#pragma unroll
        for (int j = 0; j < kBlk; ++j) {
          o[j][0] *= al[0];
          o[j][1] *= al[1];
          o[j][2] *= al[0];
          o[j][3] *= al[1];
        }
      };
      auto store_score = [&](int token, float a, float bb) {
        float* const d = srow + (long long)token * gs + 2 * tq;
        if (gs == 1) {
          if (tq == 0) *d = a;
        } else if (2 * tq < gs) {
          *reinterpret_cast<float2*>(d) = make_float2(a, bb);
        }
      };

      // NB blocks of 16 keys from block k0 of the page in stage s
      auto attend = [&](auto blocks, int k0, int s, int item) {
        constexpr int NB = decltype(blocks)::value;
        const uint32_t kb = base + s * C::kStageBytes, vb = kb + C::kTileBytes;
        const float2 sc = scale[s];
        float sr[NB][4];
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) sr[k][x] = 0.0f;
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          const uint32_t off = swz<D>(mrow, 2 * cb + mch);
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            uint32_t r[4];  // keys 16k + g4, + 8; channels 32 cb + 4 tq .., + 16
            ldsm4(kb + 16 * D * (k0 + k) + off, r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u0 = r[2 * h] ^ 0x80808080u, u1 = r[2 * h + 1] ^ 0x80808080u;
              const uint32_t a[4] = {h2_of(u0, 0x4140), h2_of(u1, 0x4140), h2_of(u0, 0x4342), h2_of(u1, 0x4342)};
              mma_f16(sr[k], a, qh[2 * cb + h].x, qh[2 * cb + h].y);
            }
          }
        }
        const float f0 = sc.x * hs[0], f1 = sc.x * hs[1];
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          sr[k][0] *= f0;
          sr[k][1] *= f1;
          sr[k][2] *= f0;
          sr[k][3] *= f1;
          mt[0] = fmaxf(mt[0], fmaxf(sr[k][0], sr[k][2]));
          mt[1] = fmaxf(mt[1], fmaxf(sr[k][1], sr[k][3]));
          store_score(item * kTile + 16 * (k0 + k) + g4, sr[k][0], sr[k][1]);
          store_score(item * kTile + 16 * (k0 + k) + g4 + 8, sr[k][2], sr[k][3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], x));
        raise(mt);
        uint32_t pb[NB][2], pl[NB][2];  // hi, lo
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float p0 = ex2(sr[k][0] - mr[0]), p1 = ex2(sr[k][1] - mr[1]);
          const float p2 = ex2(sr[k][2] - mr[0]), p3 = ex2(sr[k][3] - mr[1]);
          lr[0] += p0 + p2;
          lr[1] += p1 + p3;
          const uint32_t h01 = pack_h2(p0, p1), h23 = pack_h2(p2, p3);
          const float2 f01 = unpack_h2(h01), f23 = unpack_h2(h23);
          pb[k][0] = transpose8(h01);
          pb[k][1] = transpose8(h23);
          pl[k][0] = transpose8(pack_h2(p0 - f01.x, p1 - f01.y));
          pl[k][1] = transpose8(pack_h2(p2 - f23.x, p3 - f23.y));
        }
#pragma unroll
        for (int cb = 0; cb < D / 32; ++cb) {
          const uint32_t off = swz<D>(mrow, 2 * cb + mch);
          float acc[2][4], low[2][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[0][x] = acc[1][x] = low[0][x] = low[1][x] = 0.0f;
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            uint32_t r[4];  // channels 32 cb + 16 h + 2 g4, + 1 of keys 16k + 2 tq, + 1 (, + 8)
            ldsm4t(vb + 16 * D * (k0 + k) + off, r);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t u0 = r[2 * h] ^ 0x80808080u, u1 = r[2 * h + 1] ^ 0x80808080u;
              const uint32_t a[4] = {h2_of(u0, 0x4240), h2_of(u0, 0x4341), h2_of(u1, 0x4240), h2_of(u1, 0x4341)};
              mma_f16(acc[h], a, pb[k][0], pb[k][1]);
              mma_f16(low[h], a, pl[k][0], pl[k][1]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[2 * cb + h][x] = fmaf(acc[h][x] + low[h][x], sc.y, o[2 * cb + h][x]);
        }
      };
      for (; ok && next < seen + npage; next += SPLIT ? 1 : kCons) {
        const int s = next % C::kStages;
        const int item = i0 + next - seen;
        // Stage s last held page next - kStages.  Where that was another warp's, its release (which
        // this fill waited for) makes the full barrier's phase before this one known to be
        // complete, so the parity wait on it is exact.
        ok = (SPLIT || next < C::kStages || mbar_wait(bar_empty + s * 8, ((next / C::kStages) - 1) & 1, err)) &&
             mbar_wait(bar_full + s * 8, (next / C::kStages) & 1, err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        attend(std::integral_constant<int, SPLIT ? 1 : 4>{}, SPLIT ? warp : 0, s, item);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + s * 8);
      }
      seen += npage;

      if (i1 == st.x + 1) {
        // ---- the tail: rows 0 .. st.y - 1 of the tail buffer and the new token behind them
        const int tl = st.y;
        const long long trow = (long long)row * kTile * D, nrow = (long long)row * D;
        const int r0 = 16 * warp;
        if (r0 <= tl) {
          // key row r, or none
          auto at = [&](const uint16_t* tail, const uint16_t* fresh, int r) -> const uint16_t* {
            return r < tl ? tail + trow + (long long)r * D : r == tl ? fresh + nrow : nullptr;
          };
          const uint16_t* const ka = at(c.k_tail, p.k_new, r0 + g4);
          const uint16_t* const kb2 = at(c.k_tail, p.k_new, r0 + g4 + 8);
          float sr[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          uint2 a0[kBlk], a1[kBlk];
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            a0[j] = ka ? *reinterpret_cast<const uint2*>(ka + 16 * j + 4 * tq) : make_uint2(0, 0);
            a1[j] = kb2 ? *reinterpret_cast<const uint2*>(kb2 + 16 * j + 4 * tq) : make_uint2(0, 0);
          }
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            const uint32_t a[4] = {a0[j].x, a1[j].x, a0[j].y, a1[j].y};
            mma_b16(sr, a, qb[j].x, qb[j].y);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) sr[x] *= p.scale_log2;
          if (!ka) sr[0] = sr[1] = -INFINITY;
          if (!kb2) sr[2] = sr[3] = -INFINITY;
          if (ka) store_score(st.x * kTile + r0 + g4, sr[0], sr[1]);
          if (kb2) store_score(st.x * kTile + r0 + g4 + 8, sr[2], sr[3]);
          float mt[2] = {fmaxf(sr[0], sr[2]), fmaxf(sr[1], sr[3])};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], x));
          raise(mt);
          const float p0 = ex2(sr[0] - mr[0]), p1 = ex2(sr[1] - mr[1]);
          const float p2 = ex2(sr[2] - mr[0]), p3 = ex2(sr[3] - mr[1]);
          lr[0] += p0 + p2;
          lr[1] += p1 + p3;
          const uint32_t h01 = pack_b2(p0, p1), h23 = pack_b2(p2, p3);
          const uint32_t l01 = pack_b2(p0 - __uint_as_float(h01 << 16), p1 - __uint_as_float(h01 & 0xFFFF0000u));
          const uint32_t l23 = pack_b2(p2 - __uint_as_float(h23 << 16), p3 - __uint_as_float(h23 & 0xFFFF0000u));
          const uint32_t bh0 = transpose8(h01), bh1 = transpose8(h23), bl0 = transpose8(l01), bl1 = transpose8(l23);
          const uint16_t* vr[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) vr[x] = at(c.v_tail, p.v_new, r0 + 2 * tq + (x & 1) + 8 * (x >> 1));
          uint32_t v[kBlk][4];
#pragma unroll
          for (int j = 0; j < kBlk; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              v[j][x] = vr[x] ? *reinterpret_cast<const uint32_t*>(vr[x] + 16 * j + 2 * g4) : 0u;
#pragma unroll
          for (int j = 0; j < kBlk; ++j) {
            // channels 16 j + 2 g4 (rows g4) and + 1 (rows g4 + 8) of keys 2 tq, + 1, + 8, + 9
            const uint32_t a[4] = {__byte_perm(v[j][0], v[j][1], 0x5410), __byte_perm(v[j][0], v[j][1], 0x7632),
                                   __byte_perm(v[j][2], v[j][3], 0x5410), __byte_perm(v[j][2], v[j][3], 0x7632)};
            mma_b16(o[j], a, bh0, bh1);
            mma_b16(o[j], a, bl0, bl1);
          }
        }
        // the append: slot tl belongs to nobody else
        if (warp == 0) {
          for (int x = lane; x < D / 8; x += 32) {
            reinterpret_cast<uint4*>(c.k_tail + trow + (long long)tl * D)[x] = reinterpret_cast<const uint4*>(p.k_new + nrow)[x];
            reinterpret_cast<uint4*>(c.v_tail + trow + (long long)tl * D)[x] = reinterpret_cast<const uint4*>(p.v_new + nrow)[x];
          }
          if (lane == 0) c.pos[(long long)row * (c.cap + 1) * kTile + st.x * kTile + tl] = st.z;
        }
      }

      // ---- the four warps' states into one partial of this piece
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) lr[h] += __shfl_xor_sync(0xffffffffu, lr[h], x);
      cons_sync();  // the last row's partial has been read
      float* const rw = red + warp * GRP * (D + 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int hd = 2 * tq + h;
        if (hd < GRP) {
#pragma unroll
          for (int j = 0; j < kBlk; ++j)
            *reinterpret_cast<float2*>(rw + hd * (D + 2) + 16 * j + 2 * g4) = make_float2(o[j][h], o[j][2 + h]);
          if (g4 == 0) *reinterpret_cast<float2*>(rw + hd * (D + 2) + D) = make_float2(mr[h], lr[h]);
        }
      }
      cons_sync();
      const long long slot = (long long)blockIdx.x + row;  // (piece, row) pairs rise along the list
      if (t == 0 && i0 == 0) p.row_info[row].x = blockIdx.x;
      if (t == 0 && i1 == st.x + 1) p.row_info[row].y = blockIdx.x;
      for (int x = t; x < grp * (D / 2); x += 32 * kCons) {
        const int gg = x / (D / 2), ch = x % (D / 2) * 2;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kCons; ++w) M = fmaxf(M, red[(w * GRP + gg) * (D + 2) + D]);
        float L = 0.0f;
        float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kCons; ++w) {
          const float* const r = red + (w * GRP + gg) * (D + 2);
          const float wt = r[D] == -INFINITY ? 0.0f : ex2(r[D] - M);
          const float2 v = *reinterpret_cast<const float2*>(r + ch);
          L += r[D + 1] * wt;
          acc.x += v.x * wt;
          acc.y += v.y * wt;
        }
        const long long pi = slot * grp + gg;
        *reinterpret_cast<float2*>(p.part_o + pi * D + ch) = acc;
        if (ch == 0) *reinterpret_cast<float2*>(p.part_ml + pi * 2) = make_float2(M, L);
      }
      return true;
    });
  }
  __syncthreads();
  if (t == 0 && *err) atomicOr(p.status, *err);
}

// One CTA per (chunk of tokens, KV head, sequence).
template <int D, int GS>
__global__ void __launch_bounds__(kFinThreads, 8) paged_finish_kernel(const PagedStepParams p) {
  __shared__ float s_w[GS * kPieces];  // pieces' m, then their weights 2^(m - M) / L
  __shared__ float s_m[GS], s_il[GS];
  __shared__ float s_red[kFinThreads / 32 * D];
  const tra_paged_cache& c = p.c;
  const int x = blockIdx.x, g = blockIdx.y, b = blockIdx.z, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int row = b * c.Hkv + g, grp = c.Hq / c.Hkv;
  grid_wait();
  const int4 st = p.ws_state[b];
  const int2 info = p.row_info[row];
  const int last = p.row_info[row - g + c.Hkv - 1].y;  // last piece of the sequence
  const long long row64 = (long long)row * (c.cap + 1) * kTile;
  const int tok = st.x * kTile + st.y;  // tokens before the step
  // the row's chunk per CTA: whatever the cache's capacity, its tokens are spread over the grid
  const int chunk = max(256, ((tok + 1) / (int)gridDim.x / 128 + 1) * 128);
  if (row_items(st, c.cap) == 0) {  // idle, bad or full: the row stays
    const PagedRow kind = paged_row(st, c.cap);
    if (x == 0 && g == 0 && t == 0) {
      reinterpret_cast<int4*>(p.state_out)[b] = st;
      if (kind != kRowIdle) atomicOr(p.status, kind == kRowBad ? TRA_DEV_BAD_CACHE : TRA_DEV_CACHE_FULL);
    }
    if (kind == kRowOk && p.weight_out != c.weight)
      for (long long i = (long long)x * chunk + t; i < tok && i < (long long)(x + 1) * chunk; i += kFinThreads)
        p.weight_out[row64 + i] = c.weight[row64 + i];
    return;
  }
  const int total = tok + 1;
  if ((long long)x * chunk >= total) return;
  const int chunks = (total + chunk - 1) / chunk;
  const long long slot0 = (long long)info.x + row;
  const int cnt = info.y - info.x + 1;
  // Page numbers out of range: of this head (its output and weights stay), and, for the one CTA that
  // writes the state, of any head of the sequence (the state stays).  A sequence's slots follow one
  // another, with zeroes between.
  const bool writes_state = x == 0 && g == 0;
  const int all = writes_state ? last + c.Hkv - info.x : cnt;
  const int bad_first = t < all ? p.bad[slot0 + t] : 0;  // (on its way during the heads' loop)
  int bad_here = 0, bad_any = 0;
  for (int i = t + kFinThreads; i < all; i += kFinThreads) {
    const int v = p.bad[slot0 + i];
    if (i < cnt) bad_here |= v;
    bad_any |= v;
  }
  for (int h = warp; h < grp; h += kFinThreads / 32) {
    float M = -INFINITY, L = 0.0f;
    for (int i = lane; i < cnt; i += 32) {  // running maximum and sum over this lane's pieces
      const float2 v = *reinterpret_cast<const float2*>(p.part_ml + ((slot0 + i) * grp + h) * 2);
      s_w[h * kPieces + i] = v.x;
      if (v.x > M) {
        L *= ex2(M - v.x);
        M = v.x;
      }
      if (v.x != -INFINITY) L += v.y * ex2(v.x - M);
    }
    float MM = M;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) MM = fmaxf(MM, __shfl_xor_sync(0xffffffffu, MM, o));
    L = M == -INFINITY ? 0.0f : L * ex2(M - MM);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    const float il = 1.0f / L;
    if (lane == 0) {
      s_m[h] = MM;
      s_il[h] = il;
    }
    for (int i = lane; i < cnt; i += 32) {
      const float m = s_w[h * kPieces + i];
      s_w[h * kPieces + i] = m == -INFINITY ? 0.0f : ex2(m - MM) * il;
    }
  }
  const bool stays = __syncthreads_or(bad_here | (t < cnt ? bad_first : 0));
  if (writes_state) {
    const bool same = __syncthreads_or(bad_any | bad_first);
    if (t == 0)
      reinterpret_cast<int4*>(p.state_out)[b] =
          same ? st : make_int4(st.x + (st.y == kTile - 1), (st.y + 1) % kTile, st.z + 1, st.w);
  }
  if (stays) {
    if (p.weight_out != c.weight)
      for (long long i = (long long)x * chunk + t; i < tok && i < (long long)(x + 1) * chunk; i += kFinThreads)
        p.weight_out[row64 + i] = c.weight[row64 + i];
    return;
  }

  // outputs of heads x, x + chunks, ...: a warp takes every fourth piece, then they are joined
  for (int gg = x; gg < grp; gg += chunks) {
    constexpr int kEach = D / 32;  // channels per lane
    float acc[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int i = warp; i < cnt; i += kFinThreads / 32) {
      const float w = s_w[gg * kPieces + i];
      const float* const o = p.part_o + ((slot0 + i) * grp + gg) * D + lane * kEach;
      float v[kEach];
      if constexpr (kEach == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
#pragma unroll
      for (int k = 0; k < kEach; ++k) acc[k] += v[k] * w;
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) s_red[warp * D + lane * kEach + k] = acc[k];
    __syncthreads();
    for (int ch = t; ch < D; ch += kFinThreads) {
      float o = 0.0f;
#pragma unroll
      for (int w = 0; w < kFinThreads / 32; ++w) o += s_red[w * D + ch];
      const __nv_bfloat16 r = __float2bfloat16_rn(o);
      p.out[((long long)b * c.Hq + g * grp + gg) * D + ch] = *reinterpret_cast<const uint16_t*>(&r);
    }
    __syncthreads();
  }
  // weights: a token's probabilities over the group's heads, in order
  const float* const srow = p.scores + row64 * GS;
  const int end = (int)min((long long)total, (long long)(x + 1) * chunk);
  float hm[GS], hl[GS];  // (a padded head adds nothing)
#pragma unroll
  for (int h = 0; h < GS; ++h) {
    hm[h] = h < grp ? s_m[h] : 0.0f;
    hl[h] = h < grp ? s_il[h] : 0.0f;
  }
  // (a batch of loads before its stores: the compiler cannot tell their arrays apart)
  constexpr int kBatch = GS > 4 ? 4 : 8;
  for (int i0 = x * chunk + t; i0 < end; i0 += kBatch * kFinThreads) {
    float s[kBatch][GS], old[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kFinThreads;
      if (i >= end) break;
      const float* const src = srow + (long long)i * GS;
      if constexpr (GS % 4 == 0) {
#pragma unroll
        for (int h = 0; h < GS; h += 4) *reinterpret_cast<float4*>(s[k] + h) = *reinterpret_cast<const float4*>(src + h);
      } else if constexpr (GS % 2 == 0) {
#pragma unroll
        for (int h = 0; h < GS; h += 2) *reinterpret_cast<float2*>(s[k] + h) = *reinterpret_cast<const float2*>(src + h);
      } else {
        s[k][0] = src[0];
      }
      old[k] = i < tok ? c.weight[row64 + i] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kFinThreads;
      if (i >= end) break;
      float w = 0.0f;
#pragma unroll
      for (int h = 0; h < GS; ++h) w += ex2(s[k][h] - hm[h]) * hl[h];
      p.weight_out[row64 + i] = old[k] + w;
    }
  }
  if (x == 0 && st.y == kTile - 1) {  // the tail is full: the row's next page
    const int page = c.table[(long long)row * c.cap + st.x];
    if (page >= 0 && page < c.n_pool) {  // (a step whose waits ran out may have left no mark)
      const uint16_t* const kt = c.k_tail + (long long)row * kTile * D;
      const uint16_t* const vt = c.v_tail + (long long)row * kTile * D;
      const long long at = (long long)page * kTile * D;
      quantise_page<D, kFinThreads>([&](int r) { return kt + r * D; }, c.k8 + at, c.sk + page, s_red);
      quantise_page<D, kFinThreads>([&](int r) { return vt + r * D; }, c.v8 + at, c.sv + page, s_red + kFinThreads / 32);
    }
  }
}

template <int D, int GRP, bool SPLIT>
cudaError_t launch_step_s(const PagedStepParams& p, const PagedMaps& m, cudaStream_t s) {
  using C = StepCfg<D, GRP>;
  static SmemLimit limit;
  cudaError_t e = limit.raise(paged_step_kernel<D, GRP, SPLIT>, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_ex(paged_step_kernel<D, GRP, SPLIT>, dim3(kPieces), kStepThreads, C::kSmem, s, 0, false, p, m);
}

template <int D, int GRP>
cudaError_t launch_step_g(const PagedStepParams& p, const PagedMaps& m, cudaStream_t s) {
  // Where the cache has room for few pages per piece the warps split them (a row of 2K tokens, when
  // this came in: 11.0 -> 9.3 us; 27 pages per piece split or not by a branch in one kernel: 3 % slower than apart).
  const long long most = (long long)p.c.B * p.c.Hkv * (p.c.cap + 1);
  return most <= (long long)kSplitItems * kPieces ? launch_step_s<D, GRP, true>(p, m, s) : launch_step_s<D, GRP, false>(p, m, s);
}

template <int D>
cudaError_t launch_step_d(const PagedStepParams& p, const PagedMaps& m, cudaStream_t s) {
  const tra_paged_cache& c = p.c;
  const int grp = c.Hq / c.Hkv;
  cudaError_t e = grp <= 2 ? launch_step_g<D, 2>(p, m, s) : grp <= 4 ? launch_step_g<D, 4>(p, m, s) : launch_step_g<D, 8>(p, m, s);
  if (e != cudaSuccess) return e;
  // about one wave of CTAs over all rows (eight per SM), chunks of 256 tokens at least
  const long long most = ((long long)c.cap + 1) * kTile, rows = (long long)c.B * c.Hkv;
  const long long nx = std::min((1184 + rows - 1) / rows, (most + 255) / 256);
  const dim3 grid((unsigned)nx, c.Hkv, c.B);
  switch (paged_score_stride(grp)) {
    case 1: return launch_ex(paged_finish_kernel<D, 1>, grid, kFinThreads, 0, s, 0, true, p);
    case 2: return launch_ex(paged_finish_kernel<D, 2>, grid, kFinThreads, 0, s, 0, true, p);
    case 4: return launch_ex(paged_finish_kernel<D, 4>, grid, kFinThreads, 0, s, 0, true, p);
    case 6: return launch_ex(paged_finish_kernel<D, 6>, grid, kFinThreads, 0, s, 0, true, p);
    default: return launch_ex(paged_finish_kernel<D, 8>, grid, kFinThreads, 0, s, 0, true, p);
  }
}

}  // namespace

PagedLayout paged_layout(const tra_paged_cache& c) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t grp = c.Hq / c.Hkv, rows = (size_t)c.B * c.Hkv, slots = kPieces + rows;
  PagedLayout l{};
  // the step's arrays and the cut's share the space behind the states
  l.state = 0;
  const size_t head = up((size_t)c.B * 16);
  l.info = head;
  l.bad = l.info + up(rows * 8);
  l.ml = l.bad + up(slots * 4);
  l.o = l.ml + up(slots * grp * 8);
  l.scores = l.o + up(slots * grp * c.d * 4);
  const size_t step_end = l.scores + up(rows * (c.cap + 1) * kTile * paged_score_stride((int)grp) * 4);
  l.src = head;
  l.dst = l.src + up(rows * c.cap * kTile * 4);
  l.weight = l.dst + up(rows * c.cap * 4);
  l.pos = l.weight + up(rows * (c.cap + 1) * kTile * 4);
  const size_t cut_end = l.pos + up(rows * (c.cap + 1) * kTile * 4);
  l.total = step_end > cut_end ? step_end : cut_end;
  return l;
}

cudaError_t launch_paged_step(const PagedStepParams& p, const PagedMaps& m, cudaStream_t s) {
  return p.c.d == 128 ? launch_step_d<128>(p, m, s) : launch_step_d<64>(p, m, s);
}

}  // namespace tra
