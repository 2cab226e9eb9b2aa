// chunk_few.cu -- attention of a ragged chunk of new tokens over a paged cache
// of QJL codes: few rows (several drafted tokens, short chunks), on the
// 5th-generation tensor cores.  The operator is that of chunk_tc.cu.
//
// With few rows per (sequence, KV head) the cache is read about once per row
// tile and reading it is the bound: m/8 + 2 + 2 d bytes per key.  So nothing
// is written back in between, and everything per key is done once for all the
// rows of a tile.  The keys are the M side of both products, 128 at a time,
// and the NR (32 or 64) rows the N side, whose cost falls with the rows:
//     S^T[128 keys x NR] = Z U^T        (binary16, K = m)
//     P^T = 2^(rowscale S^T - max)      (bf16, through shared memory)
//     O^T[d x NR] += V^T P^T            (bf16, V as it lies in its pages)
// with u = S q.  Z is expanded straight into tensor memory as the A operand,
// 64 coordinates of 128 keys at a time: +-||k_t||, the stored binary16 norm
// with the code bit as its sign, so the score comes out of the product scaled.
// A 32-bit word pairs coordinates (j, j + 16) of a code word, one shift and
// one LOP3 each, and U has its coordinates in the same order.  U is binary16
// with a power-of-two scale per row (rounded by 2^-11 of each entry at most,
// random in sign).
//
// A softmax thread holds one key and all NR rows.  The rows' maxima are shared
// through shared memory and renewed only when a weight would pass 2^16 (one vote
// of the 128 threads per tile), so the common tile has no reduction at all;
// the sums (of the rounded weights, so that what they have in common cancels)
// stay with the threads until the row tile ends.
//
// Measured: 2 to 8 tokens each of 8 sequences of up to 32768 keys, 32 heads over
// 8 (d = 128, m = 256), are 0.49 GB in 120 to 125 us, 4 TB/s (attend alone 117 to 119
// from cold caches, DRAM 51% busy, issue slots 39%).  A key tile takes 1740 clocks
// of an SM where its bytes alone would take 1590; the rest of the time is prep (8
// to 12 us, latency, for all of which attend waits although its first copies need
// only the plan), the first tiles' arrival and the joining of split rows.
//
// Kernels: prep (u and the plan, chunk.cuh), attend.  Warps of attend: 0-3
// softmax and output; then 8 (4 with 64 rows) that expand, a quarter of the
// keys each and, when 8, alternate chunks; one for MMA issue and tensor memory;
// one for copies (V by a bulk tensor copy, codes and norms by a bulk copy per
// granule, whose keys lie side by side in one page).  Every wait is bounded;
// one that runs out records DERR_TC_WAIT_TIMEOUT.
#include "chunk.cuh"
#include "jl_tc.cuh"

#include <cuda_fp16.h>

namespace jlk {

using namespace tcx;
namespace chunk {
namespace {

constexpr int SM_WARPS = 4, EXP_WARP0 = SM_WARPS;
constexpr int BOX = BN * 128;      // 128 keys of 64 16-bit elements
constexpr int ZRING = 2;           // groups of Z chunks in tensor memory

// Place of coordinate i in the contraction's order (see the file's head).
__host__ __device__ __forceinline__ int k_slot(int i) {
  return (i & ~31) + 2 * (i & 15) + ((i >> 4) & 1);
}

constexpr int PREP_ROWS = 16;

// Block 0 makes the plan; the others project PREP_ROWS rows each with
// mma.sync (a few rows, where the time is one trip to memory: the sketch's
// operand registers are loaded straight from it before anything else).  A bf16
// query is one operand; an fp32 one is three bf16 ones that add up to it, so
// all products are exact and the sums fp32.  12 us for 1280 rows from cold caches.
template <int M, int D, bool F32>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(const Params p) {
  griddep_launch_dependents();  // attend may set itself up meanwhile
  if (blockIdx.x == 0) {
    make_plan(p);
    return;
  }
  constexpr int WARPS = PREP_THREADS / 32, NT = M / 8 / WARPS, KT = D / 16;
  constexpr int TERMS = F32 ? 3 : 1, LD = D + 8;
  __shared__ __align__(16) uint16_t q[TERMS][PREP_ROWS][LD];
  __shared__ float top[PREP_ROWS][WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = warp * NT * 8;                      // the warp's sketch rows
  uint32_t b[NT][KT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const uint32_t *s = reinterpret_cast<const uint32_t *>(
          p.S + (int64_t)(n0 + 8 * n + (lane >> 2)) * D + 16 * k + 2 * (lane & 3));
      b[n][k][0] = __ldg(s);
      b[n][k][1] = __ldg(s + 4);
    }
  const uint32_t rows = (uint32_t)(p.N * p.G);       // of a KV head
  const uint32_t total = rows * p.Hkv;
  const uint32_t r0 = (blockIdx.x - 1) * PREP_ROWS;
  const float sgn = p.scale < 0.f ? -1.f : 1.f;
#pragma unroll
  for (int i = threadIdx.x; i < PREP_ROWS * D; i += PREP_THREADS) {
    const uint32_t r = r0 + i / D;
    float v = 0.f;
    if (r < total) {
      const uint32_t h = r / rows, tg = r - h * rows, tok = tg / p.G, g = tg - tok * p.G;
      v = sgn * load_q(p.Q, F32, tok * p.q_tok + (int64_t)(h * p.G + g) * p.q_head + i % D);
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      const uint16_t x = __bfloat16_as_ushort(__float2bfloat16_rn(v));
      q[t][i / D][i % D] = x;
      v -= bf16_bits_to_f32(x);
    }
  }
  __syncthreads();
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
  for (int t = TERMS - 1; t >= 0; --t)               // the small terms first
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const uint16_t *x = &q[t][lane >> 2][16 * k + 2 * (lane & 3)];
      uint32_t a[4];
      a[0] = *reinterpret_cast<const uint32_t *>(x);
      a[1] = *reinterpret_cast<const uint32_t *>(x + 8 * LD);
      a[2] = *reinterpret_cast<const uint32_t *>(x + 8);
      a[3] = *reinterpret_cast<const uint32_t *>(x + 8 * LD + 8);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma_bf16_16816(acc[n], a[0], a[1], a[2], a[3], b[n][k][0], b[n][k][1]);
    }
  // the largest entry of each row: over the four lanes that hold it, the warps
  float m0 = 0.f, m1 = 0.f;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m0 = fmaxf(m0, fmaxf(fabsf(acc[n][0]), fabsf(acc[n][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(acc[n][2]), fabsf(acc[n][3])));
  }
#pragma unroll
  for (int o = 2; o; o >>= 1) {
    m0 = fmaxf(m0, __shfl_xor_sync(~0u, m0, o));
    m1 = fmaxf(m1, __shfl_xor_sync(~0u, m1, o));
  }
  if ((lane & 3) == 0) {
    top[lane >> 2][warp] = m0;
    top[(lane >> 2) + 8][warp] = m1;
  }
  __syncthreads();
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = (lane >> 2) + 8 * half;
    const uint32_t row = r0 + r;
    if (row >= total) break;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v = fmaxf(v, top[r][w]);
    const float2 f = row_power(v);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        p.w.U[(int64_t)row * M + k_slot(n0 + 8 * n + 2 * (lane & 3) + e)] =
            __half_as_ushort(__float2half_rn(acc[n][2 * half + e] * f.x));
    if (warp == 0 && (lane & 3) == 0)
      p.w.rs[row] = fmaxf((float)(1.2533141373155002512 / M * 1.4426950408889634074) *
                              fabsf(p.scale) * f.y,
                          MIN_SCALE);
  }
}

// ---------------------------------------------------------------------------
// attend

template <int K, int D, int NR>
struct Cfg {
  // warps: with 64 rows a softmax thread holds twice the scores and sums, and
  // the registers of a second set of expanding warps go to it
  static constexpr int EXP_PARTS = NR == 64 ? 1 : 2, EXP_WARPS = 4 * EXP_PARTS;
  static constexpr int MMA_WARP = EXP_WARP0 + EXP_WARPS, LOAD_WARP = MMA_WARP + 1;
  static constexpr int THREADS = (LOAD_WARP + 1) * 32;
  static constexpr int KCH = K / 64;                 // 64-coordinate chunks of 32 columns,
  static constexpr int GCH = KCH < 4 ? KCH : 4;      // handed over in groups of up to four
  static constexpr int NG = KCH / GCH, GCOLS = GCH * 32;
  static constexpr int DB = D / 64;                  // boxes of a V tile
  static constexpr int U_BYTES = KCH * NR * 128;
  static constexpr int P_ROW = NR * 2, P_BYTES = BN * P_ROW;
  static constexpr int CODE_ROW = K / 8;
  // a stage: V, codes and norms of a key tile
  static constexpr int ST_V = DB * BOX, ST_C = BN * CODE_ROW, ST_N = BN * 2;
  static constexpr int STAGE = ST_V + (ST_C + ST_N + 1023) / 1024 * 1024;
  static constexpr int SMALL = 4096;                 // row arrays and barriers
  static constexpr int FREE = 227 * 1024 - 1024 - SMALL - U_BYTES - 2 * P_BYTES;
  static constexpr int ST = FREE / STAGE > 4 ? 4 : FREE / STAGE;
  static constexpr int OFF_ST = U_BYTES;             // stages, then P: a 64-dim V's second
  static constexpr int OFF_P = OFF_ST + ST * STAGE;  // box is read past its stage
  static constexpr int OFF_SMALL = OFF_P + 2 * P_BYTES;
  static constexpr int SMEM = OFF_SMALL + SMALL + 1024;
  // tensor memory columns
  static constexpr int COL_O = 2 * NR, COL_Z = 3 * NR < 128 ? 128 : 256, TMEM = 512;
  static_assert(ST >= 2, "stages");
  static_assert(COL_Z + ZRING * GCOLS <= TMEM && COL_O + NR <= COL_Z, "tensor memory");
  static_assert(SMEM <= 227 * 1024 && 2 * P_BYTES >= BOX, "shared memory");
  static_assert(MOST_RECORDS * NR * 4 <= 2 * P_BYTES, "weights of the records that are joined");
};

// Operands whose rows lie along K (V^T: dims contiguous within a key; P^T: rows
// contiguous within a key): 128-byte (64 elements) or 64-byte (32 elements)
// swizzle, `group` bytes from 8 keys to the next 8, `box` bytes from 64 rows or
// dims to the next 64.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t box, uint32_t group,
                                            uint32_t swizzle) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(box >> 4) << 16;
  d |= (uint64_t)(group >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)swizzle << 61;
  return d;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// What the softmax threads share about the rows of a row tile.
template <int NR>
struct Rows {
  float scale[NR], neg[NR];   // of a score; minus the maximum weights refer to
  float factor[NR];           // of sums and accumulators when that is renewed
  float part[SM_WARPS][NR];   // a maximum or sum of each warp
  float total[SM_WARPS][NR];  // sums, of records that are joined
  float sum[NR];
  int seen[NR];               // keys the row sees
  int out[NR];                // row of the output
};

// The 32 values of each lane reduced over the warp: lane j gets value j's.
template <typename F>
__device__ __forceinline__ float reduce32(float (&v)[32], int lane, F f) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const bool up = lane & o;
      const float keep = up ? v[j + o] : v[j], send = up ? v[j] : v[j + o];
      v[j] = f(keep, __shfl_xor_sync(~0u, send, o));
    }
  }
  return v[0];
}

template <int K, int D, int NR>
__global__ void __launch_bounds__(Cfg<K, D, NR>::THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_u,
                  const __grid_constant__ CUtensorMap map_v, const Params p) {
  using C = Cfg<K, D, NR>;
  constexpr int EXP_PARTS = C::EXP_PARTS, EXP_WARPS = C::EXP_WARPS, MMA_WARP = C::MMA_WARP;
  extern __shared__ uint8_t chunk_smem[];
  const uint32_t raw = smem_u32(chunk_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *g = chunk_smem + (base - raw);
  Rows<NR> &rows = *reinterpret_cast<Rows<NR> *>(g + C::OFF_SMALL);
  constexpr int OFF_BAR = C::OFF_SMALL + 3584;
  static_assert(sizeof(Rows<NR>) <= 3584, "row arrays");
  const uint32_t bar0 = base + OFF_BAR;
  int nbar = 0;
  auto bars = [&](int n) {
    const uint32_t a = bar0 + 8u * nbar;
    nbar += n;
    return a;
  };
  const uint32_t full = bars(C::ST), empty = bars(C::ST), zfull = bars(ZRING), zempty = bars(ZRING),
                 sfull = bars(2), pready = bars(2), pvdone = bars(2), ufull = bars(1),
                 uempty = bars(1), ofree = bars(1), fin = bars(1);
  uint32_t *holder = reinterpret_cast<uint32_t *>(g + OFF_BAR + 496);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(g + OFF_BAR + 500);
  volatile int *join_flag = reinterpret_cast<volatile int *>(g + OFF_BAR + 504);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, EXP_WARPS + 1);  // codes read by each warp, V by the product
    }
    for (int i = 0; i < ZRING; ++i) {
      mbar_init(zfull + 8 * i, EXP_WARPS);
      mbar_init(zempty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pready + 8 * i, SM_WARPS);
      mbar_init(pvdone + 8 * i, 1);
    }
    mbar_init(ufull, 1);
    mbar_init(uempty, 1);
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
  if (warp == C::LOAD_WARP && lane == 0) {
    prefetch_map(&map_u);
    prefetch_map(&map_v);
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *holder;
  griddep_wait();  // the plan and U

  Seg s;
  bool more = seg_first(s, p);
  uint32_t it = 0, sg = 0;  // key tiles and segments (with key tiles) so far

  if (warp < SM_WARPS) {
    // ---------------- softmax: thread = key; output: thread = dim
    const int r = threadIdx.x;
    const uint32_t trow = tmem + ((uint32_t)(32 * warp) << 16);
    auto sync = []() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); };
    auto any = [](bool x) {  // of the 128 threads
      uint32_t y;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
          " bar.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(y)
          : "r"((uint32_t)x)
          : "memory");
      __syncwarp();
      return y != 0;
    };
    bool ok = true;  // the same for the 128 threads wherever they meet
    for (; more; more = seg_next(s, p)) {
      const int64_t row0 = (int64_t)s.mt * NR;                 // of the (sequence, KV head)
      const int nrow = (int)min((int64_t)NR, (int64_t)s.n * p.G - row0);
      auto token = [&](int j) { return (int)((row0 + j) / p.G); };
      if (r < NR) {
        const int64_t urow = ((int64_t)s.h * p.N + s.start) * p.G + row0 + r;
        rows.scale[r] = r < nrow ? __ldcg(p.w.rs + urow) : MIN_SCALE;
        rows.seen[r] = r < nrow ? min(s.L, max(0, s.L - s.n + token(r) + 1)) : 0;
        rows.neg[r] = 0.f;
        const int tok = token(r);
        rows.out[r] = (s.start + tok) * p.Hq + s.h * p.G + (int)(row0 + r - (int64_t)tok * p.G);
      }
      sync();
      // the first key that some row does not see
      const int all_seen = min(s.L, max(0, s.L - s.n + token(0) + 1));
      float l[NR];
#pragma unroll
      for (int j = 0; j < NR; ++j) l[j] = 0.f;
      for (int k = 0; k < s.nk; ++k, ++it) {
        const int buf = it & 1;
        if (ok) ok = wait_phase(sfull + 8 * buf, (it >> 1) & 1u, abort_flag, p.err);
        if (any(!ok)) {
          ok = false;
          break;
        }
        fence_after();
        const int t0 = (s.k0 + k) * BN, t = t0 + r;
        const uint32_t tS = trow + (uint32_t)(buf * NR);
        const bool edge = t0 + BN > all_seen;
        // 32 rows at a time: x = the scores, -inf where the row does not see
        // the key; a weight is 2^(x scale + neg)
        auto scores = [&](int j0, uint32_t (&v)[32]) {
          ld32(tS + j0, v);
          ld_wait(v);
          if (edge) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (t >= rows.seen[j0 + j]) v[j] = 0xff800000u;
          }
        };
        auto exponents = [&](int j0, uint32_t (&v)[32], float &top) {
          const float4 *sc = reinterpret_cast<const float4 *>(rows.scale + j0);
          const float4 *ng = reinterpret_cast<const float4 *>(rows.neg + j0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 a = sc[j], b = ng[j];
            const float x[4] = {fmaf(__uint_as_float(v[4 * j]), a.x, b.x),
                                fmaf(__uint_as_float(v[4 * j + 1]), a.y, b.y),
                                fmaf(__uint_as_float(v[4 * j + 2]), a.z, b.z),
                                fmaf(__uint_as_float(v[4 * j + 3]), a.w, b.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              top = fmaxf(top, x[e]);
              v[4 * j + e] = __float_as_uint(x[e]);
            }
          }
        };
        uint32_t v[NR / 32][32];
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NR / 32; ++q) {
          scores(32 * q, v[q]);
          exponents(32 * q, v[q], top);
        }
        if (any(k == 0 || top > RENEW)) {
          // the tile's maximum of each row, over the threads
#pragma unroll
          for (int q = 0; q < NR / 32; ++q) {
            scores(32 * q, v[q]);
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[q][j]);
            rows.part[warp][32 * q + lane] =
                reduce32(x, lane, [](float a, float b) { return fmaxf(a, b); });
          }
          sync();
          if (r < NR) {
            float x = fmaxf(fmaxf(rows.part[0][r], rows.part[1][r]),
                            fmaxf(rows.part[2][r], rows.part[3][r]));
            x = x == -INFINITY ? x : x * rows.scale[r];
            const float old = -rows.neg[r];
            // a row without a key so far refers to 0
            const float now = k == 0 ? (x == -INFINITY ? 0.f : x) : fmaxf(old, x);
            rows.factor[r] = k == 0 || now == old ? 1.f : fast_exp2(old - now);
            rows.neg[r] = -now;
          }
          sync();
          if (k > 0) {
            // earlier products must have landed before the accumulator is scaled
            if (ok) ok = wait_phase(pvdone + 8 * ((it - 1) & 1u), ((it - 1) >> 1) & 1u, abort_flag,
                                    p.err);
            if (any(!ok)) {
              ok = false;
              break;
            }
            fence_after();
#pragma unroll
            for (int q = 0; q < NR / 16; ++q) {
              uint32_t o[16];
              ld16(trow + C::COL_O + 16 * q, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float f = rows.factor[16 * q + j];
                o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                l[16 * q + j] *= f;
              }
              st16(trow + C::COL_O + 16 * q, o);
            }
            st_wait();
          }
#pragma unroll
          for (int q = 0; q < NR / 32; ++q) exponents(32 * q, v[q], top);
        }
        // weights, in the order of the operand: row j of key t at element j
        uint8_t *P = g + C::OFF_P + buf * C::P_BYTES + r * C::P_ROW;
        const int swz = NR == 64 ? (r & 7) : ((r >> 1) & 3);
#pragma unroll
        for (int q = 0; q < NR / 32; ++q)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 8 * u + 2 * e;
              const float a = fast_exp2(__uint_as_float(v[q][j])),
                          b = fast_exp2(__uint_as_float(v[q][j + 1]));
              w[e] = pack_bf16x2(a, b);
              // the sums are of the rounded weights: what they have in common cancels
              l[32 * q + j] += __uint_as_float(w[e] << 16);
              l[32 * q + j + 1] += __uint_as_float(w[e] & 0xffff0000u);
            }
            *reinterpret_cast<uint4 *>(P + (((4 * q + u) ^ swz) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        // values of keys past the last one, whatever their page holds there,
        // must not meet a weight of zero
        if (t >= s.L) {  // (the tile's copies have landed: its scores are there)
          uint8_t *V = g + C::OFF_ST + (it % C::ST) * C::STAGE + value_offset(r, p, D);
          for (int x = 0; x < C::DB; ++x)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4 *>(V + x * p.gran * 128 + 16 * e) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready + 8 * buf);
      }
      if (!ok) break;
      if (s.nk > 0) {
        ok = wait_phase(pvdone + 8 * ((it - 1) & 1u), ((it - 1) >> 1) & 1u, abort_flag, p.err);
        if (any(!ok)) {
          ok = false;
          break;
        }
        fence_after();
      }
      // sums over the threads
#pragma unroll
      for (int q = 0; q < NR / 32; ++q) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = l[32 * q + j];
        rows.part[warp][32 * q + lane] =
            reduce32(x, lane, [](float a, float b) { return a + b; });
      }
      sync();
      if (r < NR)
        rows.sum[r] = (rows.part[0][r] + rows.part[1][r]) + (rows.part[2][r] + rows.part[3][r]);
      sync();
      const bool whole = s.k0 == 0 && s.k1 == s.units;
      auto write = [&](int j, float x) {  // dim r of row j
        const float sum = rows.sum[j];
        const float y = sum == 0.f ? 0.f : __fdividef(x, sum);
        if (JL_IN_RANGE(p.err, rows.out[j], 1, p.N * p.Hq))
          p.out[(int64_t)rows.out[j] * D + r] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
      };
      // states of a split row tile: [NR][d + 2]
      const Split split(s, p);
      float *mine = p.w.part + split.record(blockIdx.x) * (int64_t)(NR * (D + 2));
      const bool mine_ok = JL_IN_RANGE(p.err, split.record(blockIdx.x), 1, 2 * SM_COUNT);
#pragma unroll
      for (int q = 0; q < NR / 16; ++q) {
        if (16 * q >= nrow) break;
        uint32_t o[16] = {};
        if (s.nk > 0) ld16(trow + C::COL_O + 16 * q, o);
        if (r < D) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int j = 16 * q + e;
            if (j >= nrow) break;
            if (whole)
              write(j, __uint_as_float(o[e]));
            else if (mine_ok)
              mine[j * (D + 2) + r] = __uint_as_float(o[e]);
          }
        }
      }
      if (s.nk > 0) {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree);
      }
      if (!whole) {
        if (r < nrow && mine_ok)
          *reinterpret_cast<float2 *>(mine + r * (D + 2) + D) =
              make_float2(-rows.neg[r], rows.sum[r]);
        if (last_to_arrive(split, p, 0, 1, SM_WARPS * 32, r == 0, join_flag)) {
          // the joined maximum and sum of each row: a quarter of the records
          // (half with 64 rows) to each group of NR threads
          auto record = [&](int64_t c) {
            return p.w.part + split.record(c) * (int64_t)(NR * (D + 2));
          };
          constexpr int GR = SM_WARPS * 32 / NR;
          const int j = r % NR, gr = r / NR;
          auto state = [&](int64_t c) {
            return j < nrow && c <= split.c1
                       ? __ldcg(reinterpret_cast<const float2 *>(record(c) + j * (D + 2) + D))
                       : make_float2(-INFINITY, 0.f);
          };
          auto join = [](float2 a, float2 b) {
            const float m = fmaxf(a.x, b.x);
            if (m == -INFINITY) return make_float2(m, a.y + b.y);
            return make_float2(m, (a.y == 0.f ? 0.f : a.y * fast_exp2(a.x - m)) +
                                      (b.y == 0.f ? 0.f : b.y * fast_exp2(b.x - m)));
          };
          float2 ms = make_float2(-INFINITY, 0.f);
          for (int64_t c = split.c0 + gr; c <= split.c1; c += GR) {
            const float2 x = state(c);
            if (x.y != 0.f) ms = join(ms, x);
          }
          rows.part[gr][j] = ms.x;
          rows.total[gr][j] = ms.y;
          sync();
          if (r < NR) {
            ms = make_float2(rows.part[0][r], rows.total[0][r]);
            for (int q = 1; q < GR; ++q)
              ms = join(ms, make_float2(rows.part[q][r], rows.total[q][r]));
            rows.neg[r] = -ms.x;
            rows.sum[r] = ms.y;
          }
          // each record's weight for each row, where P lies (nobody reads or
          // writes it until this warp's next tile)
          float *weight = reinterpret_cast<float *>(g + C::OFF_P);
          const int records = (int)(split.c1 - split.c0) + 1;
          sync();
          for (int i = r; i < records * NR; i += SM_WARPS * 32) {
            const float2 x = state(split.c0 + i / NR);  // (i % NR is j)
            weight[i] = x.y == 0.f ? 0.f : fast_exp2(x.x + rows.neg[j]);
          }
          sync();
          // the accumulators of eight rows, their loads side by side
          if (r < D) {
            for (int j0 = 0; j0 < nrow; j0 += 8) {
              float o[8] = {};
#pragma unroll 2
              for (int i = 0; i < records; ++i) {
                const float *acc = record(split.c0 + i) + r;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  asm volatile("ld.global.cg.f32 %0, [%1];\n"
                               : "=f"(y[e])
                               : "l"(acc + min(j0 + e, nrow - 1) * (D + 2)));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float w = weight[i * NR + j0 + e];
                  o[e] = w == 0.f ? o[e] : fmaf(w, y[e], o[e]);
                }
              }
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (j0 + e < nrow) write(j0 + e, o[e]);
            }
          }
        }
      }
      sync();  // the row arrays are free for the next row tile
    }
  } else if (warp < MMA_WARP) {
    // ---------------- expand: quarter q of the keys, chunks pt, pt + EXP_PARTS, ..
    const int q = warp & 3, pt = (warp - EXP_WARP0) >> 2;
    const int r = 32 * q + lane;
    constexpr int KP = (C::GCH + EXP_PARTS - 1) / EXP_PARTS;  // of a group
    const uint32_t tz = tmem + ((uint32_t)(32 * q) << 16) + C::COL_Z;
    bool ok = true;
    for (; ok && more; more = seg_next(s, p)) {
      for (int k = 0; ok && k < s.nk; ++k, ++it) {
        const uint32_t st = it % C::ST;
        if (!wait_phase(full + 8 * st, (it / C::ST) & 1u, abort_flag, p.err)) {
          ok = false;
          break;
        }
        const uint8_t *stage = g + C::OFF_ST + st * C::STAGE + C::ST_V;
        uint2 w[C::NG * KP];
#pragma unroll
        for (int i = 0; i < C::NG * KP; ++i) {
          const int kc = (i / KP) * C::GCH + pt + EXP_PARTS * (i % KP);
          if (pt + EXP_PARTS * (i % KP) < C::GCH)
            w[i] = *reinterpret_cast<const uint2 *>(stage + r * C::CODE_ROW + 8 * kc);
        }
        const uint32_t n16 = *reinterpret_cast<const uint16_t *>(stage + C::ST_C + 2 * r);
        const uint32_t key = 0x80008000u ^ (n16 << 16 | n16);  // bit set: +norm
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * st);
#pragma unroll
        for (int gr = 0; gr < C::NG; ++gr) {
          const uint32_t c = it * C::NG + gr, slot = c % ZRING;
          if (!wait_phase(zempty + 8 * slot, ((c / ZRING) & 1u) ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          fence_after();  // the products that read this slot before
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            const int kc = pt + EXP_PARTS * i;
            if (kc >= C::GCH) break;
            const uint2 x = w[gr * KP + i];
            uint32_t z[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              z[j] = ((x.x << (15 - j)) & 0x80008000u) ^ key;
              z[16 + j] = ((x.y << (15 - j)) & 0x80008000u) ^ key;
            }
            st32(tz + C::GCOLS * slot + 32 * kc, z);
          }
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(zfull + 8 * slot);
        }
      }
    }
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issue: scores run one tile ahead of values
    constexpr uint32_t id_s = idesc_f16(BN, NR, 0);
    constexpr uint32_t id_o = idesc_f16(BN, NR, 1) | (1u << 15) | (1u << 16);
    constexpr uint32_t P_GROUP = 8 * C::P_ROW, P_SWZ = NR == 64 ? 2u : 4u;
    const uint64_t du0 = desc_sw128(base);
    // (with 64 dims the upper half of the product reads whatever follows, as
    // dims that are not there; nothing looks at it)
    const uint64_t dv0 = desc_mn(base + C::OFF_ST, p.gran * 128, 1024, 2);
    const uint64_t dp0 = desc_mn(base + C::OFF_P, BOX, P_GROUP, P_SWZ);
    uint32_t voff[BN / 16];  // of 16 keys each, in descriptor units
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk) voff[kk] = value_offset(16 * kk, p, D) >> 4;
    bool ok = true;
    uint32_t zc = 0;
    auto wait = [&](uint32_t bar, uint32_t ph) {
      const bool w = __all_sync(~0u, wait_phase(bar, ph, abort_flag, p.err));
      fence_after();
      return w;
    };
    auto scores = [&](uint32_t t) {
      for (int gr = 0; gr < C::NG; ++gr, ++zc) {
        const uint32_t slot = zc % ZRING;
        if (!wait(zfull + 8 * slot, (zc / ZRING) & 1u)) return false;
        if (elect_one()) {
          const uint32_t d = tmem + (t & 1u) * NR, z = tmem + C::COL_Z + C::GCOLS * slot;
          const uint64_t du = du0 + (uint64_t)((gr * C::GCH * NR * 128) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4 * C::GCH; ++kk)
            mma_ts(d, z + 8 * kk, du + (uint64_t)(((kk >> 2) * NR * 128 + (kk & 3) * 32) >> 4),
                   id_s, (gr | kk) ? 1u : 0u);
          commit(zempty + 8 * slot);
          if (gr == C::NG - 1) commit(sfull + 8 * (t & 1u));
        }
        __syncwarp();
      }
      return true;
    };
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      if (!(ok = wait(ufull, sg & 1u))) break;
      if (!(ok = scores(it))) break;
      for (int k = 0; k < s.nk; ++k, ++it) {
        if (k + 1 < s.nk) {
          if (!(ok = scores(it + 1))) break;
        } else {
          if (elect_one()) commit(uempty);  // U has been read
          __syncwarp();
        }
        const uint32_t st = it % C::ST;
        if (k == 0 && sg > 0 && !(ok = wait(ofree, (sg - 1) & 1u))) break;
        if (!(ok = wait(pready + 8 * (it & 1u), (it >> 1) & 1u))) break;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ss(tmem + C::COL_O,
                   dv0 + (uint64_t)((st * C::STAGE) >> 4) + voff[kk],
                   dp0 + (uint64_t)(((it & 1u) * C::P_BYTES + kk * 2 * P_GROUP) >> 4), id_o,
                   (k > 0 || kk > 0) ? 1u : 0u);
          commit(empty + 8 * st);
          commit(pvdone + 8 * (it & 1u));
        }
        __syncwarp();
      }
      ++sg;
    }
    // every product has landed before the tensor memory is given back
    if (elect_one()) commit(fin);
    __syncwarp();
    drain_wait(fin, 0);
  } else {
    // ---------------- copies: U of a segment; V, codes and norms of each key tile
    bool ok = true;
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      if (sg > 0 && !__all_sync(~0u, wait_phase(uempty, (sg - 1) & 1u, abort_flag, p.err))) break;
      if (lane == 0) {
        mbar_expect_tx(ufull, C::U_BYTES);
        const int64_t row = ((int64_t)s.h * p.N + s.start) * p.G + (int64_t)s.mt * NR;
        for (int kc = 0; kc < C::KCH; ++kc)
          tma_load_2d(base + kc * NR * 128, &map_u, kc * 64, (int)row, ufull);
      }
      __syncwarp();
      ++sg;
      // lane i copies granule i; the next tile's page is looked up meanwhile
      auto place = [&](int k, bool &here) -> int64_t {
        const int t = (s.k0 + k) * BN + p.gran * lane;
        here = k < s.nk && lane < BN >> p.gran_log && t < s.L;
        return here ? ((int64_t)page_of(p, s.b, t) * p.Hkv + s.h) * p.P + t % p.P : 0;
      };
      bool here;
      int64_t row = place(0, here);
      for (int k = 0; k < s.nk; ++k) {
        const uint32_t st = it % C::ST;
        const int grans = __popc(__ballot_sync(~0u, here));
        if (!__all_sync(~0u, wait_phase(empty + 8 * st, ((it / C::ST) & 1u) ^ 1u, abort_flag,
                                        p.err))) {
          ok = false;
          break;
        }
        const uint32_t bytes_v = p.gran * D * 2, bytes_c = p.gran * C::CODE_ROW,
                       bytes_n = p.gran * 2;
        const uint32_t bar = full + 8 * st;
        if (lane == 0) mbar_expect_tx(bar, grans * (bytes_v + bytes_c + bytes_n));
        __syncwarp();
        if (here) {
          const uint32_t dst = base + C::OFF_ST + st * C::STAGE;
          bulk_load(dst + C::ST_V + lane * bytes_c, p.codes + row * (K / 32), bytes_c, bar);
          bulk_load(dst + C::ST_V + C::ST_C + lane * bytes_n, p.norms + row, bytes_n, bar);
          tma_load_3d(dst + lane * bytes_v, &map_v, 0, (int)row, 0, bar);
        }
        __syncwarp();
        ++it;
        row = place(k + 1, here);
      }
    }
    if (*abort_flag) {  // let the copies in flight land before the block leaves
      if (sg > 0) drain_wait(ufull, (sg - 1) & 1u);
      for (uint32_t i = it > C::ST ? it - C::ST : 0; i < it; ++i)
        drain_wait(full + 8 * (i % C::ST), (i / C::ST) & 1u);
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

template <int M, int D, int NR>
cudaError_t launch_nr(const Params &p, const ChunkArgs &a, cudaStream_t stream) {
  using C = Cfg<M, D, NR>;
  CUtensorMap map_u, map_v;
  const int64_t rows = p.N * p.Hq;
  if (!tc::make_map(&map_u, p.w.U, rows, M, M, NR) ||
      !make_value_map(&map_v, a.value_pages, (uint64_t)p.num_pages * p.Hkv * p.P, D, p.gran))
    return cudaErrorInvalidValue;
  const int64_t prep = 1 + (rows + PREP_ROWS - 1) / PREP_ROWS;
  auto prep_k = a.q_f32 ? prep_kernel<M, D, true> : prep_kernel<M, D, false>;
  prep_k<<<(unsigned)prep, PREP_THREADS, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attend_kernel<M, D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_after(attend_kernel<M, D, NR>, p.blocks, C::THREADS, C::SMEM, stream, map_u, map_v,
                      p);
}

template <int M, int D>
cudaError_t launch_t(const Params &p, const ChunkArgs &a, cudaStream_t stream) {
  return p.rows == 32 ? launch_nr<M, D, 32>(p, a, stream) : launch_nr<M, D, 64>(p, a, stream);
}

}  // namespace

// 32 rows where the sequences have that many on average, 64 where they have
// more: the products and weights of rows that are not there cost as much.
int few_rows(int64_t N, int B, int G) {
  return N * G <= (int64_t)FEW_ROWS_LEAST * B ? FEW_ROWS_LEAST : FEW_ROWS_MOST;
}

size_t few_workspace(int64_t N, int B, int Hq, int Hkv, int m, int d, Work *w, void *base) {
  const int rows = few_rows(N, B, Hq / Hkv);
  return lay_out(w, base, N, B, Hq, Hkv, rows, m, (size_t)rows * (d + 2), 0);
}

cudaError_t launch_few(Params p, const ChunkArgs &a, cudaStream_t stream) {
  p.rows = few_rows(p.N, p.B, p.G);
  few_workspace(p.N, p.B, p.Hq, p.Hkv, a.m, a.d, &p.w, a.workspace);
#define JL_CASE(MM, DD) \
  if (a.m == MM && a.d == DD) return launch_t<MM, DD>(p, a, stream);
  JL_CASE(64, 64) JL_CASE(128, 64) JL_CASE(256, 64) JL_CASE(512, 64)
  JL_CASE(64, 128) JL_CASE(128, 128) JL_CASE(256, 128) JL_CASE(512, 128)
#undef JL_CASE
  return cudaErrorNotSupported;
}

}  // namespace chunk

// Which kernel: expanding the keys costs what one reading and one writing of
// 2 d bytes per key cost and then makes a row cheap, so it pays from about
// MANY rows per (sequence, KV head) on, and only while the expanded keys stay
// inside MAX_KEYS bytes of workspace.  Microseconds here / there, 4 sequences of 8
// KV heads, bf16 queries, all sequences with as many rows and keys:
//   d, m, G      rows   512 keys   2048      8192        32768
//   128, 256, 4   128    40 / 32   60 / 46    98 / 100   225 / 253
//                 160    57 / 35   68 / 49   119 / 106   303 / 270
//                 512    89 / 38  120 / 64   246 / 134   794 / 423
//   64, 128, 1    128    32 / 30   52 / 41    80 / 77    200 / 211
//                 160    42 / 34   58 / 42    99 / 83    276 / 228
//                 512    73 / 32   93 / 52   206 / 109   664 / 339
// m = 128 at d = 128 and m = 64 at d = 64, G = 4 turn at the same rows.  Below 160
// rows and 8192 keys the rule takes the slower one, by up to a quarter.  It goes by
// the average over the batch, padding rows included, and decides for all of it: a
// chunk of 2048 tokens beside 31 single ones over 32768 keys each takes 2916 us
// in one call, 1627 as two (beside 63 over 8192: 1170 and 527).
constexpr int MANY = 160;
constexpr int64_t MAX_KEYS = (int64_t)8 << 30;
static bool many(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int d) {
  const int64_t tiles = (max_len + chunk::BN - 1) / chunk::BN * B * Hkv;
  return N * (Hq / Hkv) >= (int64_t)MANY * B && tiles * chunk::BN * d * 2 <= MAX_KEYS &&
         tiles < ((int64_t)1 << 31) / chunk::BN;
}

bool chunk_sizes_fit(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int d) {
  constexpr int64_t most = ((int64_t)1 << 31) - 1;
  if (max_len > most + 1 - chunk::BN) return false;  // a length rounded up to a tile
  // a sequence has at most this many row tiles, each of at most all key tiles
  const int G = Hq / Hkv;
  const int rows = many(N, B, Hq, Hkv, max_len, d) ? chunk::MANY_ROWS : chunk::few_rows(N, B, G);
  return (N * G / rows + 1) * ((max_len + chunk::BN - 1) / chunk::BN) <= most;
}

size_t chunk_workspace_bytes(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int m, int d) {
  return many(N, B, Hq, Hkv, max_len, d)
             ? chunk::many_workspace(N, B, Hq, Hkv, max_len, d, nullptr, nullptr)
             : chunk::few_workspace(N, B, Hq, Hkv, m, d, nullptr, nullptr);
}

// The most that shapes up to these need: of either kernel's parts the larger, with
// the expanded keys of as many sequences as `many` lets in.
size_t chunk_workspace_bound(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int m, int d) {
  const int64_t most = N * (Hq / Hkv) / MANY, seqs = B < most ? B : most;
  const int64_t tiles = (max_len + chunk::BN - 1) / chunk::BN * seqs * Hkv;
  const int64_t tile = (int64_t)chunk::BN * d * 2;
  const int64_t keys = tiles < MAX_KEYS / tile ? tiles * tile : MAX_KEYS;
  const int rows = seqs > 0 ? chunk::MANY_ROWS : chunk::FEW_ROWS_MOST;
  return chunk::lay_out(nullptr, nullptr, N, B, Hq, Hkv, chunk::FEW_ROWS_LEAST, m > d ? m : d,
                        (size_t)rows * (d + 2), (size_t)keys);
}

cudaError_t launch_chunk(const ChunkArgs &a, cudaStream_t stream) {
  chunk::Params p{};
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidSymbol;
  p.codes = a.sign_pages; p.norms = a.norm_pages;
  p.table = a.block_table; p.cu = a.cu_seqlens; p.lens = a.seq_lens;
  p.Q = a.Q; p.q_tok = a.q_tok; p.q_head = a.q_head; p.S = a.S; p.out = a.out;
  p.B = a.B; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.P = a.page_tokens;
  p.max_pages = a.max_pages; p.num_pages = a.num_pages; p.N = a.N; p.max_len = a.max_len;
  p.key_tiles = (int)((a.max_len + chunk::BN - 1) / chunk::BN);
  p.gran_log = a.page_tokens % 128 == 0 ? 7 : a.page_tokens % 64 == 0 ? 6 : 5;
  p.gran = 1 << p.gran_log;
  p.scale = a.softmax_scale;
  const int sms = device_sm_count();
  p.blocks = sms < chunk::SM_COUNT ? sms : chunk::SM_COUNT;
  return many(a.N, a.B, a.Hq, a.Hkv, a.max_len, a.d) ? chunk::launch_many(p, a, stream)
                                                     : chunk::launch_few(p, a, stream);
}

}  // namespace jlk
