// chunk_tc.cu -- attention of a ragged chunk of new tokens over a paged cache
// of QJL codes, on the 5th-generation tensor cores.
//
// Sequence b brings n_b tokens whose keys are already in its cache of L_b
// keys; token i sees the keys t < L_b - n_b + i + 1.  With
//     s(q, k_t) = sqrt(pi/2)/m * ||k_t|| * <S q, z_t>,   z_t = +-1 code bits
// (the estimator of decode) the result is softmax over the seen keys of
// softmax_scale * s, applied to the bf16 values; a token that sees no key
// gets zeros.
//
// Rows.  The query heads of a KV head share its keys, so row i * G + g of a
// (sequence, KV head) is token i, head g; 128 consecutive rows make the M side
// of one tile of work and 128 keys its N side.
//
// Kernels, on one stream:
//   1. prep     u = S q per row, as binary16 with a power-of-two scale per
//               row (its largest entry lies in [2^13, 2^14)), and the plan:
//               lengths checked, work counted in key tiles.
//   2. attend   a fixed grid; each block takes an equal run of the key tiles
//               of all (sequence, KV head, row tile) in order, so a long
//               context with few rows is split and many rows are balanced,
//               causal triangle included.  A row tile that lies in one block
//               is written out, a split one leaves softmax states.
//   3. combine  joins the states of split row tiles.
//
// attend, per key tile (all products fp32-accumulated in tensor memory):
//     S[128 rows x 128 keys] = U Z^T       (binary16, K = m)
//     P = 2^(rowscale ||k_t|| S - max)     (bf16, back into tensor memory)
//     O[128 x d] += P V                    (bf16, V as it lies in its pages)
// Z is expanded from the code bits into shared memory, 64 coordinates of 128
// keys at a time: a 32-bit word pairs coordinates (j, j + 16) of a code word,
// one shift and one LOP3 each, and U has its coordinates in the same order.
// P is rounded to bf16 (half a step, 2^-9 of each weight, against values that
// are bf16 themselves); its sum is taken before the rounding, in fp32.
//
// The maximum is renewed only when a row's grows by more than 2^8: until then
// weights up to 2^8 are as exact, and the accumulator in tensor memory need
// not be rescaled.
//
// Warps: 0-3 softmax (one row per thread) and output, 4 MMA issue and tensor
// memory, 5 copies (U and V by bulk tensor copies, a 32-key granule of V lies
// in one page), 6-9 expand (one key per thread, codes two tiles ahead).
// Every wait is bounded; one that runs out records DERR_TC_WAIT_TIMEOUT.
#include "jl_common.cuh"
#include "jl_internal.h"
#include "jl_tc.cuh"

#include <cuda_fp16.h>

namespace jlk {

using namespace tcx;
namespace chunk {

constexpr int BM = 128, BN = 128;  // rows and keys of a tile
constexpr int GRAN = 32;           // keys that surely share a page
constexpr int SM_WARPS = 4, MMA_WARP = 4, LOAD_WARP = 5, EXP_WARP0 = 6, EXP_WARPS = 4;
constexpr int THREADS = (EXP_WARP0 + EXP_WARPS) * 32;
constexpr int BOX = BM * 128;      // 128 rows of 64 16-bit elements
constexpr float RENEW = 8.f;       // log2 growth of a row's maximum that renews it
constexpr int SN = 2;              // norm stages

// The plan, made on the device from the call's lengths.
struct Plan {
  int64_t total;      // units (key tiles, at least one per row tile)
  int64_t quota;      // units per block
};
struct Work {         // workspace
  Plan *plan;
  int64_t *b_unit;    // [B + 1] first unit of each sequence
  int32_t *b_tile;    // [B] first entry of its row tiles in mt_pre
  int32_t *start, *count, *len;  // [B] first row, tokens, keys, made safe
  int32_t *mt_pre;    // per sequence: units before each row tile of a head, and their sum
  uint16_t *U;        // [Hkv][N G][m] binary16
  float *rs;          // [Hkv][N G] row scale
  float *part;        // [2 blocks][128][d + 2] softmax states
};

struct Params {
  Work w;
  const uint32_t *codes;
  const uint16_t *norms;
  const int32_t *table, *cu, *lens;
  const void *Q;
  int64_t q_tok, q_head;
  const uint16_t *S;
  uint16_t *out;
  int B, Hq, Hkv, G, P, max_pages, num_pages, blocks, min_units;
  int64_t N, max_len;
  float scale;        // softmax_scale
  int *err;
};

// ---------------------------------------------------------------------------
// prep

constexpr int PREP_THREADS = 256, PREP_ROWS = 16;

// Units of row tile mt: key tiles that its last token sees, at least one.
__device__ __forceinline__ int tile_units(int mt, int n, int L, int G) {
  const int last = min(n - 1, (BM * mt + BM - 1) / G);
  const int seen = max(0, L - n + last + 1);
  return max(1, (seen + BN - 1) / BN);
}

__device__ void make_plan(const Params &p) {
  __shared__ int64_t units[PREP_THREADS];  // of a head, then before the sequence
  __shared__ int tiles[PREP_THREADS];
  __shared__ int first[PREP_THREADS], tokens[PREP_THREADS];
  __shared__ int64_t u_done;
  __shared__ int t_done, rows_done;
  if (threadIdx.x == 0) {
    u_done = 0;
    t_done = rows_done = 0;
  }
  for (int b0 = 0; b0 < p.B; b0 += PREP_THREADS) {
    const int b = b0 + threadIdx.x;
    int n = 0, L = 0, nt = 0;
    int64_t c0 = 0, tot = 0;
    if (b < p.B) {
      c0 = p.cu[b];
      const int64_t c1 = p.cu[b + 1], l = p.lens[b];
      if (c0 < 0 || c1 < c0 || c1 > p.N) {
        record_device_error(p.err, DERR_DECODE_PLAN);
        c0 = 0;
      } else {
        n = (int)(c1 - c0);
      }
      if (l < 0 || l > p.max_len) record_device_error(p.err, DERR_DECODE_PLAN);
      L = (int)(l < 0 ? 0 : l > p.max_len ? p.max_len : l);
      nt = (int)(((int64_t)n * p.G + BM - 1) / BM);
      for (int mt = 0; mt < nt; ++mt) tot += tile_units(mt, n, L, p.G);
    }
    units[threadIdx.x] = tot;
    tiles[threadIdx.x] = nt ? nt + 1 : 0;
    first[threadIdx.x] = (int)c0;
    tokens[threadIdx.x] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
      int64_t u = u_done;
      int t = t_done, rows = rows_done;
      for (int i = 0; i < PREP_THREADS && b0 + i < p.B; ++i) {
        if (tokens[i] && first[i] < rows) {  // rows that an earlier sequence has
          record_device_error(p.err, DERR_DECODE_PLAN);
          tokens[i] = tiles[i] = 0;
          units[i] = 0;
        }
        if (tokens[i]) rows = first[i] + tokens[i];
        const int64_t x = units[i];
        const int y = tiles[i];
        units[i] = u;
        tiles[i] = t;
        u += x * p.Hkv;
        t += y;
      }
      u_done = u;
      t_done = t;
      rows_done = rows;
    }
    __syncthreads();
    if (b < p.B) {
      n = tokens[threadIdx.x];
      if (n == 0) nt = 0;
      p.w.b_unit[b] = units[threadIdx.x];
      p.w.b_tile[b] = tiles[threadIdx.x];
      p.w.start[b] = (int32_t)c0;
      p.w.count[b] = n;
      p.w.len[b] = L;
      int32_t *pre = p.w.mt_pre + tiles[threadIdx.x];
      int u = 0;
      for (int mt = 0; mt < nt; ++mt) {
        pre[mt] = u;
        u += tile_units(mt, n, L, p.G);
      }
      if (nt) pre[nt] = u;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.w.b_unit[p.B] = u_done;
    int64_t q = (u_done + p.blocks - 1) / p.blocks;
    if (q < p.min_units) q = p.min_units;
    p.w.plan->total = u_done;
    p.w.plan->quota = q;
  }
}

// Place of coordinate i in the contraction's order (see the file's head).
__host__ __device__ __forceinline__ int k_slot(int i) {
  return (i & ~31) + 2 * (i & 15) + ((i >> 4) & 1);
}

// The power of two that brings a row whose largest entry is `top` into
// [2^13, 2^14), as (2^e, 2^-e); 1 for a row of zeros, infinities or NaN.
__device__ __forceinline__ float2 row_power(float top) {
  if (!(top > 0.f) || isinf(top)) return make_float2(1.f, 1.f);
  int e;
  frexpf(top, &e);  // top = f 2^e, f in [1/2, 1)
  e = 14 - e;
  e = max(-120, min(120, e));
  return make_float2(ldexpf(1.f, e), ldexpf(1.f, -e));
}

__device__ __forceinline__ float load_q(const void *Q, bool f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float *>(Q) + i)
             : bf16_bits_to_f32(__ldg(static_cast<const uint16_t *>(Q) + i));
}

// Block 0 makes the plan; the others project PREP_ROWS rows each.  A thread
// holds one sketch row in registers and meets every query row in shared
// memory (a broadcast), m threads side by side.
template <int M, int D, bool F32>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(const Params p) {
  if (blockIdx.x == 0) {
    make_plan(p);
    return;
  }
  __shared__ __align__(16) float q[PREP_ROWS][D];
  __shared__ float top[PREP_ROWS][PREP_THREADS / 32];
  const int64_t rows = p.N * p.G;                    // of a KV head
  const int64_t total = rows * p.Hkv;
  const int64_t r0 = (int64_t)(blockIdx.x - 1) * PREP_ROWS;
  const float sgn = p.scale < 0.f ? -1.f : 1.f;
  for (int i = threadIdx.x; i < PREP_ROWS * D; i += PREP_THREADS) {
    const int64_t r = r0 + i / D;
    float v = 0.f;
    if (r < total) {
      const int h = (int)(r / rows);
      const int64_t tg = r - h * rows, tok = tg / p.G;
      const int g = (int)(tg - tok * p.G);
      v = sgn * load_q(p.Q, F32, tok * p.q_tok + (int64_t)(h * p.G + g) * p.q_head + i % D);
    }
    q[i / D][i % D] = v;
  }
  __syncthreads();
  // SPLIT threads groups share the rows when m < 256; m = 512 takes two passes
  constexpr int TH = M < PREP_THREADS ? M : PREP_THREADS;
  constexpr int PASS = M / TH, GROUPS = PREP_THREADS / TH, RG = PREP_ROWS / GROUPS;
  const int grp = threadIdx.x / TH;
  float acc[PASS][RG];
#pragma unroll
  for (int ps = 0; ps < PASS; ++ps) {
    const int i = threadIdx.x % TH + ps * TH;
#pragma unroll
    for (int r = 0; r < RG; ++r) acc[ps][r] = 0.f;
    const uint4 *s = reinterpret_cast<const uint4 *>(p.S + (int64_t)i * D);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 w = __ldg(s + c);
      const float x[8] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                          __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u),
                          __uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u),
                          __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u)};
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        const float4 a = *reinterpret_cast<const float4 *>(&q[grp * RG + r][8 * c]);
        const float4 b = *reinterpret_cast<const float4 *>(&q[grp * RG + r][8 * c + 4]);
        float t = acc[ps][r];
        t = fmaf(a.x, x[0], t); t = fmaf(a.y, x[1], t);
        t = fmaf(a.z, x[2], t); t = fmaf(a.w, x[3], t);
        t = fmaf(b.x, x[4], t); t = fmaf(b.y, x[5], t);
        t = fmaf(b.z, x[6], t); t = fmaf(b.w, x[7], t);
        acc[ps][r] = t;
      }
    }
  }
  // the largest entry of each row: over the row's warps
  constexpr int RW = TH / 32;  // warps of a row group
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    float v = 0.f;
#pragma unroll
    for (int ps = 0; ps < PASS; ++ps) v = fmaxf(v, fabsf(acc[ps][r]));
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    if ((threadIdx.x & 31) == 0) top[grp * RG + r][(threadIdx.x % TH) >> 5] = v;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RG; ++r) {
    const int64_t row = r0 + grp * RG + r;
    if (row >= total) break;
    float v = 0.f;
    for (int w = 0; w < RW; ++w) v = fmaxf(v, top[grp * RG + r][w]);
    const float2 f = row_power(v);
#pragma unroll
    for (int ps = 0; ps < PASS; ++ps)
      p.w.U[row * M + k_slot(threadIdx.x % TH + ps * TH)] =
          __half_as_ushort(__float2half_rn(acc[ps][r] * f.x));
    if (threadIdx.x % TH == 0)
      p.w.rs[row] = (float)(1.2533141373155002512 / M * 1.4426950408889634074) * fabsf(p.scale) *
                    f.y;
  }
}

// ---------------------------------------------------------------------------
// attend

// A block's run of units, one row tile after another.
struct Seg {
  int b, h, mt, nt;   // sequence, KV head, row tile, row tiles of the sequence
  int k0, k1, units;  // its units [k0, k1) of `units`
  int n, L, start;    // the sequence's tokens, keys, first row
  int nk;             // key tiles to do: 0 where the row tile sees no key
  int64_t u, end;     // next unit, end of the run
};

__device__ __forceinline__ void seg_fill(Seg &s, const Params &p) {
  const int32_t *pre = p.w.mt_pre + __ldg(p.w.b_tile + s.b);
  const int a = __ldg(pre + s.mt), z = __ldg(pre + s.mt + 1);
  s.units = z - a;
  const int64_t left = s.end - s.u;
  s.k1 = (int)(left < s.units - s.k0 ? s.k0 + left : s.units);
  const int last = min(s.n - 1, (BM * s.mt + BM - 1) / p.G);
  s.nk = s.L - s.n + last + 1 > 0 ? s.k1 - s.k0 : 0;
}
__device__ __forceinline__ void seg_seq(Seg &s, const Params &p) {
  s.n = __ldg(p.w.count + s.b);
  s.L = __ldg(p.w.len + s.b);
  s.start = __ldg(p.w.start + s.b);
  s.nt = (int)(((int64_t)s.n * p.G + BM - 1) / BM);
}
// First segment of the block; false when it has none.
__device__ bool seg_first(Seg &s, const Params &p) {
  const int64_t total = __ldg(&p.w.plan->total), quota = __ldg(&p.w.plan->quota);
  s.u = (int64_t)blockIdx.x * quota;
  s.end = s.u + quota < total ? s.u + quota : total;
  if (s.u >= total) return false;
  int lo = 0, hi = p.B;  // the last b whose first unit is not above u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.w.b_unit + mid) <= s.u) lo = mid; else hi = mid;
  }
  s.b = lo;
  seg_seq(s, p);
  const int64_t u0 = __ldg(p.w.b_unit + lo);
  const int64_t per_head = (__ldg(p.w.b_unit + lo + 1) - u0) / p.Hkv;
  s.h = (int)((s.u - u0) / per_head);
  const int rem = (int)(s.u - u0 - s.h * per_head);
  const int32_t *pre = p.w.mt_pre + __ldg(p.w.b_tile + lo);
  int a = 0, z = s.nt;
  while (z - a > 1) {
    const int mid = (a + z) >> 1;
    if (__ldg(pre + mid) <= rem) a = mid; else z = mid;
  }
  s.mt = a;
  s.k0 = rem - __ldg(pre + a);
  seg_fill(s, p);
  return true;
}
__device__ bool seg_next(Seg &s, const Params &p) {
  s.u += s.k1 - s.k0;
  if (s.u >= s.end) return false;
  s.k0 = 0;
  if (++s.mt == s.nt) {
    s.mt = 0;
    if (++s.h == p.Hkv) {
      s.h = 0;
      do {
        ++s.b;
        seg_seq(s, p);
      } while (s.n == 0);
    }
  }
  seg_fill(s, p);
  return true;
}

// Page of the granule that holds key t; a page outside the pool is recorded
// and replaced by page 0.
__device__ __forceinline__ int page_of(const Params &p, int b, int t) {
  const int col = t / p.P;
  int page = col < p.max_pages ? __ldg(p.table + (int64_t)b * p.max_pages + col) : -1;
  if (page < 0 || page >= p.num_pages) {
    record_device_error(p.err, DERR_PAGE);
    page = 0;
  }
  return page;
}

template <int K, int D>
struct Cfg {
  static constexpr int KCH = K / 64;               // 64-coordinate chunks of U and Z
  static constexpr int VB = D / 64;                // boxes of a V tile
  static constexpr int SV = 2, NS = 2;             // V stages, score buffers
  static constexpr int FIX = KCH * BOX + SV * VB * BOX + SN * BN * 4 + 512 + 1024;
  static constexpr int RZ_RAW = (227 * 1024 - FIX) / BOX;
  static constexpr int RZ = RZ_RAW > 8 ? 8 : RZ_RAW;  // Z chunks in flight
  static constexpr int OFF_Z = KCH * BOX;
  static constexpr int OFF_V = OFF_Z + RZ * BOX;
  static constexpr int OFF_N = OFF_V + SV * VB * BOX;
  static constexpr int OFF_BAR = OFF_N + SN * BN * 4;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;  // + align slack
  // tensor memory columns: scores, accumulator, weights (two bf16 a column).
  // The weights have columns of their own: products are ordered against each
  // other only where they share an accumulator, so the scores of a later tile
  // may not be written over weights that an issued product still reads.
  static constexpr int TMEM = 512, COL_O = NS * BN, COL_P = COL_O + D;
  static_assert(RZ >= 2, "Z ring");
  static_assert(COL_P + NS * BN / 2 <= TMEM, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// V operand: keys along K in rows of 128 bytes (64 dims), 8-key groups 1024
// bytes apart (stride offset), 64-dim boxes BOX bytes apart (leading offset),
// 128-byte swizzle.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)((uint32_t)BOX >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

template <int K, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_u,
                  const __grid_constant__ CUtensorMap map_v, const Params p) {
  using C = Cfg<K, D>;
  extern __shared__ uint8_t chunk_smem[];
  const uint32_t raw = smem_u32(chunk_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *g = chunk_smem + (base - raw);
  const uint32_t bar0 = base + C::OFF_BAR;
  int nbar = 0;
  auto bars = [&](int n) {
    const uint32_t a = bar0 + 8u * nbar;
    nbar += n;
    return a;
  };
  const uint32_t zfull = bars(C::RZ), zempty = bars(C::RZ), vfull = bars(C::SV),
                 vempty = bars(C::SV), sfull = bars(C::NS), pready = bars(C::NS),
                 nfree = bars(SN), nfull = bars(SN), ufull = bars(1), uempty = bars(1),
                 pvdone = bars(2), ofree = bars(1), fin = bars(1);
  // two barriers for the value products in turn: whoever waits for a tile's
  // knows that the tile two before it is done, not that the one before is
  auto pv_bar = [&](uint32_t t) { return pvdone + 8 * (t & 1u); };
  auto pv_phase = [](uint32_t t) { return (t >> 1) & 1u; };
  uint32_t *holder = reinterpret_cast<uint32_t *>(g + C::OFF_BAR + 496);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(g + C::OFF_BAR + 500);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::RZ; ++i) {
      mbar_init(zfull + 8 * i, EXP_WARPS);
      mbar_init(zempty + 8 * i, 1);
    }
    for (int i = 0; i < C::SV; ++i) {
      mbar_init(vfull + 8 * i, 1);
      mbar_init(vempty + 8 * i, 1);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pready + 8 * i, SM_WARPS);
    }
    for (int i = 0; i < SN; ++i) {
      mbar_init(nfree + 8 * i, SM_WARPS);
      mbar_init(nfull + 8 * i, EXP_WARPS);
    }
    mbar_init(ufull, 1);
    mbar_init(uempty, 1);
    mbar_init(pvdone, 1);
    mbar_init(pvdone + 8, 1);
    mbar_init(ofree, SM_WARPS);
    mbar_init(fin, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
        "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::"r"(smem_u32(holder)),
        "n"(C::TMEM)
        : "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *holder;
  griddep_wait();  // the plan and U

  Seg s;
  bool more = seg_first(s, p);
  uint32_t it = 0;  // key tiles of earlier segments
  uint32_t sg = 0;  // segments with key tiles so far

  if (warp < SM_WARPS) {
    // ---------------- softmax: thread = row
    const int r = threadIdx.x;
    const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16);
    bool ok = true;
    for (; ok && more; more = seg_next(s, p)) {
      const int64_t row = (int64_t)s.mt * BM + r;           // of the (sequence, KV head)
      const bool live = row < (int64_t)s.n * p.G;
      const int tok = live ? (int)(row / p.G) : 0;
      const int seen = live ? min(s.L, max(0, s.L - s.n + tok + 1)) : 0;
      const int64_t urow = ((int64_t)s.h * p.N + s.start) * p.G + row;
      const float rs = live ? __ldg(p.w.rs + urow) : 0.f;
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < s.nk; ++k, ++it) {
        const int buf = it % C::NS;
        const uint32_t sph = (it / C::NS) & 1u;
        const int ns = it % SN;
        const uint32_t tS = trow + (uint32_t)(buf * BN);
        if (!wait_phase(nfull + 8 * ns, (it / SN) & 1u, abort_flag, p.err) ||
            !wait_phase(sfull + 8 * buf, sph, abort_flag, p.err)) {
          ok = false;
          break;
        }
        __syncwarp();
        fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) ld32(tS + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) ld_wait(v[c]);
        // x = ||k_t|| * <u, z_t>; keys the row does not see are -inf
        const float4 *nrm = reinterpret_cast<const float4 *>(g + C::OFF_N + ns * BN * 4);
        const int t0 = (s.k0 + k) * BN;
        const int lim = seen - t0;  // columns the row sees
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 f = nrm[c * 8 + j];
            const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = 32 * c + 4 * j + e;
              float x = __uint_as_float(v[c][4 * j + e]) * ff[e];
              if (col >= lim) x = -INFINITY;
              top = fmaxf(top, x);
              v[c][4 * j + e] = __float_as_uint(x);
            }
          }
        const float cand = top == -INFINITY ? -INFINITY : top * rs;
        if (k == 0) {
          m = cand;
        } else {
          const bool grow = cand > m + RENEW || (m == -INFINITY && cand > m);
          if (__any_sync(~0u, grow)) {
            // earlier products must have landed before the accumulator is scaled
            if (!wait_phase(pv_bar(it - 1), pv_phase(it - 1), abort_flag, p.err)) {
              ok = false;
              break;
            }
            __syncwarp();
            fence_after();
            const float mn = grow ? cand : m;
            const float f = m == mn ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              ld32(trow + C::COL_O + c, o);
              ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              st32(trow + C::COL_O + c, o);
            }
            st_wait();
          }
        }
        const float mm = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int cc = c + (e >> 4), j = 2 * (e & 15);
            const float a = fast_exp2(fmaf(__uint_as_float(v[cc][j]), rs, -mm));
            const float b = fast_exp2(fmaf(__uint_as_float(v[cc][j + 1]), rs, -mm));
            sum += a + b;
            w[e] = pack_bf16x2(a, b);
          }
          st32(trow + (uint32_t)(C::COL_P + buf * (BN / 2) + 16 * c), w);
        }
        l += sum;
        st_wait();
        // values of keys past the last one, whatever their page holds there,
        // must not meet a weight of zero
        const int left = s.L - t0;
        if (left < BN) {
          const int vs = it % C::SV;
          if (!wait_phase(vfull + 8 * vs, (it / C::SV) & 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint8_t *V = g + C::OFF_V + vs * C::VB * BOX;
          if (r >= left)
            for (int x = 0; x < C::VB; ++x)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4 *>(V + x * BOX + r * 128 + 16 * e) =
                    make_uint4(0, 0, 0, 0);
          fence_async_smem();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(nfree + 8 * ns);
          mbar_arrive(pready + 8 * buf);
        }
      }
      if (!ok) break;
      // output: the row itself, or its state where the row tile is split
      const bool whole = s.k0 == 0 && s.k1 == s.units;
      if (s.nk > 0) {
        if (!wait_phase(pv_bar(it - 1), pv_phase(it - 1), abort_flag, p.err)) {
          ok = false;
          break;
        }
        __syncwarp();
        fence_after();
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const int64_t otok = s.start + tok;
      uint16_t *out = p.out + (otok * p.Hq + s.h * p.G + (row - (int64_t)tok * p.G)) * D;
      float *part = p.w.part +
                    ((int64_t)(2 * blockIdx.x + (s.k0 == 0 ? 1 : 0)) * BM + r) * (D + 2);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (s.nk > 0) {
          ld32(trow + C::COL_O + c, o);
          ld_wait(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (live && whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 q;
            uint32_t *qq = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float a = __uint_as_float(o[8 * e + 2 * x]),
                          b = __uint_as_float(o[8 * e + 2 * x + 1]);
              qq[x] = inv == 0.f ? 0u : pack_bf16x2(a * inv, b * inv);
            }
            *reinterpret_cast<uint4 *>(out + c + 8 * e) = q;
          }
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            *reinterpret_cast<float2 *>(part + c + e) =
                make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
        }
      }
      if (live && !whole) *reinterpret_cast<float2 *>(part + D) = make_float2(m, l);
      if (s.nk > 0) {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree);
      }
    }
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issue: scores run one tile ahead of values
    constexpr uint32_t id_s = idesc_f16(BM, BN, 0);
    constexpr uint32_t id_o = idesc_f16(BM, D, 1) | (1u << 16);  // B along its N side
    const uint64_t du0 = desc_sw128(base), dz0 = desc_sw128(base + C::OFF_Z);
    const uint64_t dv0 = desc_v(base + C::OFF_V);
    bool ok = true;
    uint32_t zc = 0;
    auto wait = [&](uint32_t bar, uint32_t ph) {
      const bool w = __all_sync(~0u, wait_phase(bar, ph, abort_flag, p.err));
      fence_after();
      return w;
    };
    // scores of key tile t (counted over all segments) into its buffer
    auto scores = [&](uint32_t t) {
      const uint32_t d = tmem + (t % C::NS) * BN;
      for (int kc = 0; kc < C::KCH; ++kc, ++zc) {
        const uint32_t st = zc % C::RZ;
        if (!wait(zfull + 8 * st, (zc / C::RZ) & 1u)) return false;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(d, du0 + (uint64_t)((kc * BOX + kk * 32) >> 4),
                   dz0 + (uint64_t)((st * BOX + kk * 32) >> 4), id_s, (kc | kk) ? 1u : 0u);
          commit(zempty + 8 * st);
        }
        __syncwarp();
      }
      if (elect_one()) commit(sfull + 8 * (t % C::NS));
      __syncwarp();
      return true;
    };
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      ok = wait(ufull, sg & 1u);
      if (ok) ok = scores(it);
      for (int k = 0; ok && k < s.nk; ++k, ++it) {
        if (k + 1 < s.nk) {
          if (!(ok = scores(it + 1))) break;
        } else {
          if (elect_one()) commit(uempty);  // U has been read
          __syncwarp();
        }
        const int vs = it % C::SV;
        if (k == 0 && sg > 0 && !(ok = wait(ofree, (sg - 1) & 1u))) break;
        if (!(ok = wait(vfull + 8 * vs, (it / C::SV) & 1u))) break;
        if (!(ok = wait(pready + 8 * (it % C::NS), (it / C::NS) & 1u))) break;
        if (elect_one()) {
          const uint32_t tp = tmem + C::COL_P + (it % C::NS) * (BN / 2);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tmem + C::COL_O, tp + 8 * kk,
                   dv0 + (uint64_t)((vs * C::VB * BOX + kk * 2048) >> 4), id_o,
                   (k > 0 || kk > 0) ? 1u : 0u);
          commit(vempty + 8 * vs);
          commit(pv_bar(it));
        }
        __syncwarp();
      }
      ++sg;
    }
    // every product has landed before the tensor memory is given back
    if (elect_one()) commit(fin);
    __syncwarp();
    drain_wait(fin, 0);
  } else if (warp == LOAD_WARP) {
    // ---------------- copies: U of a segment, V of each key tile
    bool ok = true;
    uint32_t issued = 0;
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      if (sg > 0 && !__all_sync(~0u, wait_phase(uempty, (sg - 1) & 1u, abort_flag, p.err))) break;
      if (lane == 0) {
        mbar_expect_tx(ufull, C::KCH * BOX);
        const int64_t row = ((int64_t)s.h * p.N + s.start) * p.G + (int64_t)s.mt * BM;
        for (int kc = 0; kc < C::KCH; ++kc)
          tma_load_2d(base + kc * BOX, &map_u, kc * 64, (int)row, ufull);
      }
      __syncwarp();
      ++sg;
      for (int k = 0; k < s.nk; ++k, ++it) {
        const int vs = it % C::SV;
        const int t = (s.k0 + k) * BN + GRAN * (lane & 3);
        const bool here = lane < 4 && t < s.L;
        const int page = here ? page_of(p, s.b, t) : 0;
        const int grans = __popc(__ballot_sync(~0u, here));
        if (!__all_sync(~0u, wait_phase(vempty + 8 * vs, ((it / C::SV) & 1u) ^ 1u, abort_flag,
                                        p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_expect_tx(vfull + 8 * vs, grans * GRAN * 128 * C::VB);
        __syncwarp();
        if (here) {
          const int64_t vrow = ((int64_t)page * p.Hkv + s.h) * p.P + t % p.P;
          for (int x = 0; x < C::VB; ++x)
            tma_load_2d(base + C::OFF_V + (vs * C::VB + x) * BOX + lane * GRAN * 128, &map_v,
                        64 * x, (int)vrow, vfull + 8 * vs);
        }
        __syncwarp();
        issued = it + 1;
      }
    }
    if (*abort_flag) {  // let the copies in flight land before the block leaves
      if (sg > 0) drain_wait(ufull, (sg - 1) & 1u);
      for (uint32_t i = issued > C::SV ? issued - C::SV : 0; i < issued; ++i)
        drain_wait(vfull + 8 * (i % C::SV), (i / C::SV) & 1u);
    }
  } else {
    // ---------------- expand: thread = key of the tile
    constexpr int W = K / 32;
    const int r = threadIdx.x - EXP_WARP0 * 32;
    const int swz = r & 7;
    bool ok = true;
    uint32_t zc = 0;
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      // pool row of key r of tile k; keys past the last one take the last one's
      auto pool_row = [&](int k) -> int64_t {
        if (k >= s.nk) k = s.nk - 1;
        int t = (s.k0 + k) * BN + r;
        if (t >= s.L) t = s.L - 1;
        return ((int64_t)page_of(p, s.b, t) * p.Hkv + s.h) * p.P + t % p.P;
      };
      uint32_t c[3][W];
      uint16_t nn[3];
      auto fetch = [&](int64_t row, uint32_t (&w)[W], uint16_t &n) {
        if constexpr (W >= 4) {
#pragma unroll
          for (int i = 0; i < W / 4; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p.codes + row * W) + i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
          }
        } else {
          const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p.codes + row * W));
          w[0] = x.x; w[1] = x.y;
        }
        n = __ldg(p.norms + row);
      };
      fetch(pool_row(0), c[0], nn[0]);
      fetch(pool_row(1), c[1], nn[1]);
      int64_t ahead = pool_row(2);
      for (int k = 0; k < s.nk; ++k, ++it) {
        fetch(ahead, c[2], nn[2]);
        ahead = pool_row(k + 3);
        const int ns = it % SN;
        if (!wait_phase(nfree + 8 * ns, ((it / SN) & 1u) ^ 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        reinterpret_cast<float *>(g + C::OFF_N + ns * BN * 4)[r] =
            __half2float(__ushort_as_half(nn[0]));
        __syncwarp();
        if (lane == 0) mbar_arrive(nfull + 8 * ns);
#pragma unroll
        for (int kc = 0; kc < C::KCH; ++kc, ++zc) {
          const uint32_t st = zc % C::RZ;
          if (!wait_phase(zempty + 8 * st, ((zc / C::RZ) & 1u) ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint8_t *z = g + C::OFF_Z + st * BOX + r * 128;
#pragma unroll
          for (int u = 0; u < 8; ++u) {  // pairs 4 (u % 4) .. of code word u / 4
            const uint32_t w = c[0][2 * kc + (u >> 2)];
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = ((w << (15 - (4 * (u & 3) + e))) & 0x80008000u) ^ 0xBC00BC00u;
            *reinterpret_cast<uint4 *>(z + ((u ^ swz) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(zfull + 8 * st);
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          c[0][i] = c[1][i];
          c[1][i] = c[2][i];
        }
        nn[0] = nn[1];
        nn[1] = nn[2];
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                 "n"(C::TMEM)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// combine: one warp per (row, query head) of a split row tile

constexpr int CMB_WARPS = 8;

template <int D>
__global__ void __launch_bounds__(CMB_WARPS * 32) combine_kernel(const Params p) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * CMB_WARPS + (threadIdx.x >> 5);
  const int64_t tok = id / p.Hq;
  const int hq = (int)(id - tok * p.Hq);
  if (tok >= p.N) return;
  // the sequence of the row: the last b whose first row is not above it (cu,
  // not the checked starts, which are not in order where cu is not)
  if (tok < __ldg(p.cu) || tok >= __ldg(p.cu + p.B)) return;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= tok) lo = mid; else hi = mid;
  }
  const int b = lo, n = __ldg(p.w.count + b);
  const int64_t i = tok - __ldg(p.w.start + b);
  if (i < 0 || i >= n) return;
  const int h = hq / p.G;
  const int64_t row = i * p.G + (hq - h * p.G);
  const int mt = (int)(row / BM), r = (int)(row - (int64_t)mt * BM);
  const int32_t *pre = p.w.mt_pre + __ldg(p.w.b_tile + b);
  const int64_t u0 = __ldg(p.w.b_unit + b);
  const int64_t per_head = (__ldg(p.w.b_unit + b + 1) - u0) / p.Hkv;
  const int64_t a = u0 + h * per_head + __ldg(pre + mt);
  const int64_t z = u0 + h * per_head + __ldg(pre + mt + 1);
  const int64_t quota = __ldg(&p.w.plan->quota);
  const int64_t c0 = a / quota, c1 = (z - 1) / quota;
  if (c0 == c1) return;  // one block wrote the row
  constexpr int E = D / 32;
  float m = -INFINITY, l = 0.f, o[E] = {};
  for (int64_t c = c0; c <= c1; ++c) {
    const float *part = p.w.part + ((2 * c + (c * quota <= a ? 1 : 0)) * BM + r) * (D + 2);
    const float2 ml = *reinterpret_cast<const float2 *>(part + D);
    if (ml.y == 0.f) continue;
    const float mn = fmaxf(m, ml.x);
    const float f = m == mn ? 1.f : fast_exp2(m - mn), w = fast_exp2(ml.x - mn);
    l = l * f + ml.y * w;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *reinterpret_cast<const float2 *>(part + lane * E + e);
      o[e] = o[e] * f + x.x * w;
      o[e + 1] = o[e + 1] * f + x.y * w;
    }
    m = mn;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint32_t *out = reinterpret_cast<uint32_t *>(p.out + (tok * p.Hq + hq) * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    out[e / 2] = inv == 0.f ? 0u : pack_bf16x2(o[e] * inv, o[e + 1] * inv);
}

// ---------------------------------------------------------------------------
// host

constexpr int SM_COUNT = 148;  // bounds the workspace per shape

struct Sizes {
  size_t plan, b_unit, b_tile, seq, mt_pre, U, rs, part, total;
};
static Sizes sizes(int64_t N, int B, int Hq, int Hkv, int m, int d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const int G = Hq / Hkv;
  Sizes z{};
  z.plan = up(sizeof(Plan));
  z.b_unit = up((size_t)(B + 1) * 8);
  z.b_tile = up((size_t)B * 4);
  z.seq = up((size_t)B * 4);
  z.mt_pre = up(((size_t)N * G / BM + 2 * (size_t)B + 1) * 4);
  z.U = up((size_t)N * Hq * m * 2);
  z.rs = up((size_t)N * Hq * 4);
  z.part = up((size_t)2 * SM_COUNT * BM * (d + 2) * 4);
  z.total = z.plan + z.b_unit + z.b_tile + 3 * z.seq + z.mt_pre + z.U + z.rs + z.part;
  return z;
}

template <typename... Args>
static cudaError_t launch_after(void (*kernel)(Args...), int64_t grid, int threads, size_t smem,
                                cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int M, int D>
static cudaError_t launch_t(Params p, bool f32, const uint16_t *values, cudaStream_t stream) {
  using C = Cfg<M, D>;
  CUtensorMap map_u, map_v;
  const int64_t rows = p.N * p.Hq;
  if (!tc::make_map(&map_u, p.w.U, rows, M, M, BM) ||
      !tc::make_map(&map_v, values, (uint64_t)p.num_pages * p.Hkv * p.P, D, D, GRAN))
    return cudaErrorInvalidValue;
  const int64_t prep = 1 + (rows + PREP_ROWS - 1) / PREP_ROWS;
  if (f32)
    prep_kernel<M, D, true><<<(unsigned)prep, PREP_THREADS, 0, stream>>>(p);
  else
    prep_kernel<M, D, false><<<(unsigned)prep, PREP_THREADS, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attend_kernel<M, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_after(attend_kernel<M, D>, p.blocks, THREADS, C::SMEM, stream, map_u, map_v, p);
  if (e != cudaSuccess) return e;
  return launch_after(combine_kernel<D>, (rows + CMB_WARPS - 1) / CMB_WARPS, CMB_WARPS * 32, 0,
                      stream, p);
}

}  // namespace chunk

size_t chunk_workspace_bytes(int64_t N, int B, int Hq, int Hkv, int64_t, int m, int d) {
  return chunk::sizes(N, B, Hq, Hkv, m, d).total;
}

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t stream) {
  chunk::Params p{};
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidSymbol;
  const chunk::Sizes z = chunk::sizes(a.N, a.B, a.Hq, a.Hkv, a.m, a.d);
  uint8_t *w = static_cast<uint8_t *>(a.workspace);
  auto take = [&](size_t n) {
    uint8_t *x = w;
    w += n;
    return x;
  };
  p.w.plan = reinterpret_cast<chunk::Plan *>(take(z.plan));
  p.w.b_unit = reinterpret_cast<int64_t *>(take(z.b_unit));
  p.w.b_tile = reinterpret_cast<int32_t *>(take(z.b_tile));
  p.w.start = reinterpret_cast<int32_t *>(take(z.seq));
  p.w.count = reinterpret_cast<int32_t *>(take(z.seq));
  p.w.len = reinterpret_cast<int32_t *>(take(z.seq));
  p.w.mt_pre = reinterpret_cast<int32_t *>(take(z.mt_pre));
  p.w.U = reinterpret_cast<uint16_t *>(take(z.U));
  p.w.rs = reinterpret_cast<float *>(take(z.rs));
  p.w.part = reinterpret_cast<float *>(take(z.part));
  p.codes = a.sign_pages; p.norms = a.norm_pages;
  p.table = a.block_table; p.cu = a.cu_seqlens; p.lens = a.seq_lens;
  p.Q = a.Q; p.q_tok = a.q_tok; p.q_head = a.q_head; p.S = a.S; p.out = a.out;
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.P = a.page_tokens;
  p.max_pages = a.max_pages; p.num_pages = a.num_pages; p.N = a.N; p.max_len = a.max_len;
  p.scale = a.softmax_scale;
  const int sms = device_sm_count();
  p.blocks = sms < chunk::SM_COUNT ? sms : chunk::SM_COUNT;
  p.min_units = 2;
#define JL_CASE(MM, DD) \
  if (a.m == MM && a.d == DD) return chunk::launch_t<MM, DD>(p, a.q_f32, a.value_pages, stream);
  JL_CASE(64, 64) JL_CASE(128, 64) JL_CASE(256, 64) JL_CASE(512, 64)
  JL_CASE(64, 128) JL_CASE(128, 128) JL_CASE(256, 128) JL_CASE(512, 128)
#undef JL_CASE
  return cudaErrorNotSupported;
}

}  // namespace jlk
