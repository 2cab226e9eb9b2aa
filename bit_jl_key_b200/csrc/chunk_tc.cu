// chunk_tc.cu -- attention of a ragged chunk of new tokens over a paged cache
// of QJL codes: many rows, on the 5th-generation tensor cores.
//
// Sequence b brings n_b tokens whose keys are already in its cache of L_b
// keys; token i sees the keys t < L_b - n_b + i + 1.  With
//     khat_t = sqrt(pi/2)/m * ||k_t|| * S^T z_t,   z_t = +-1 code bits,
// the estimator of decode is s(q, k_t) = <q, khat_t>, and the result is the
// softmax over the seen keys of softmax_scale * s, applied to the bf16
// values; a token that sees no key gets zeros.
//
// Where a key meets many rows it pays to map its code back once: the scores
// then contract d entries instead of m, and every operand is copied by TMA.
//
// Kernels, on one stream:
//   1. prep     the queries as binary16 with a power-of-two scale per row (its
//               largest entry lies in [2^13, 2^14): a bf16 query stays exact
//               down to 2^-20 of the row's largest), and the plan.
//   2. expand   khat as binary16, from the pages (dequant_tc.cu).
//   3. attend   the products, below.
//
// attend takes 256 rows at a time as two halves of 128, and per key tile and
// half (all products fp32-accumulated in tensor memory):
//     S[128 x 128] = Q K^T                    (binary16)
//     P = 2^(rowscale S - max)                (bf16, over the first half of each
//                                              64 keys' own columns of S)
//     O[128 x d] += P V                       (bf16, V as it lies in its pages)
// While one half is in its softmax the other's products run: the exponentials
// (16 a clock and SM) take as long as the products, so the two units share
// the time.  A half's next scores lie over the weights of its tile before, so
// they are issued once the product that reads those has landed: order is
// guaranteed only between products with one accumulator and shape, which these
// two are not.  (Issued without that wait, 3% faster, results were the same.)
// P is rounded to bf16 (half a step, 2^-8 of each weight, against values that
// are bf16 themselves).  Its sum, in fp32, is of the rounded weights, so that
// what all the weights of a row have in common cancels: a row that one key
// dominates loses nothing.
//
// A row's weights refer to the maximum of the first tile it met until one would
// pass 2^RENEW (the two threads of a row vote on it, once a tile): floating
// point keeps them as exact, and the accumulator need hardly ever be rescaled.
//
// Measured: 2048 tokens of 32 heads over 32768 keys of 8 (d = 128) are 1.07
// TFLOP of products in 1.06 to 1.24 ms, 1.00 to 0.86 PFLOP/s, the latter once the
// power limit holds the clock down; over 8192 keys attend alone takes 272 us,
// tensor pipe 47% busy, exponential unit 36%, issue slots 48%.  What bounds it is
// the round trip of a half's tile: of 2.8 us (two halves in turn) about 1.0 is
// softmax (maximum 0.25, vote 0.1, weights 0.65), 0.55 the half's two products,
// S at the rate shared memory feeds its operands, and 1.2 the handing over
// between the warps and the tensor core.  Scores ahead in parts of 64 keys, which
// hide the round trip, cost more in narrow products than they hide (d = 128: 258
// to 342 us, when the whole took that).
//
// Warps: 0-7 and 8-15 softmax and output of a half, two threads per row (64 of
// a tile's keys each: a thread alone is held up by its own latencies), 16 MMA
// issue and tensor memory, 17 copies (a granule of V lies in one page).
// Every wait is bounded; one that runs out records DERR_TC_WAIT_TIMEOUT.
#include "chunk.cuh"
#include "jl_tc.cuh"

#include <cuda_fp16.h>

namespace jlk {

using namespace tcx;
namespace chunk {
namespace {

constexpr int BM = 128, HALVES = 2, ROWS = BM * HALVES;
static_assert(ROWS == MANY_ROWS, "rows of a row tile");
constexpr int SM_WARPS = 8;                       // of a half: four for each 64 of the keys
constexpr int MMA_WARP = SM_WARPS * HALVES, LOAD_WARP = MMA_WARP + 1;
constexpr int THREADS = (LOAD_WARP + 1) * 32;
constexpr int POLY_EVERY = 4;                     // one pair of weights in so many on the FMA pipe
constexpr int BOX = BM * 128;                     // 128 rows of 64 16-bit elements

// Block 0 makes the plan; the others convert the queries, d / 8 lanes per row
// (VEC: 16 bytes at a time, where every row starts on 16 bytes).  11 us for 65536
// rows, beside the expansion.
template <int D, bool F32, bool VEC>
__global__ void __launch_bounds__(PREP_THREADS) prep_kernel(const Params p) {
  griddep_launch_dependents();  // the keys may be expanded meanwhile
  if (blockIdx.x == 0) {
    make_plan(p);
    return;
  }
  constexpr int LANES = D / 8;
  const uint32_t rows = (uint32_t)(p.N * p.Hq);
  const int lane = threadIdx.x % LANES;
  const float sgn = p.scale < 0.f ? -1.f : 1.f;
  for (uint32_t r = (blockIdx.x - 1) * (PREP_THREADS / LANES) + threadIdx.x / LANES; r < rows;
       r += (gridDim.x - 1) * (PREP_THREADS / LANES)) {
    const uint32_t tok = r / p.Hq, hq = r - tok * p.Hq, h = hq / p.G;
    const int64_t q0 = tok * p.q_tok + (int64_t)hq * p.q_head + 8 * lane;
    float q[8], top = 0.f;
    if constexpr (VEC && F32) {
      const float4 *x = reinterpret_cast<const float4 *>(static_cast<const float *>(p.Q) + q0);
      const float4 a = __ldg(x), b = __ldg(x + 1);
      q[0] = a.x; q[1] = a.y; q[2] = a.z; q[3] = a.w;
      q[4] = b.x; q[5] = b.y; q[6] = b.z; q[7] = b.w;
    } else if constexpr (VEC) {
      const uint4 x =
          __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.Q) + q0));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        q[2 * e] = __uint_as_float(w[e] << 16);
        q[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = load_q(p.Q, F32, q0 + e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(q[e]));
    // (the row's lanes leave the loop together)
    const unsigned mask = LANES == 32 ? ~0u : ((1u << LANES) - 1u) << (threadIdx.x & 31 & -LANES);
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
    const float2 f = row_power(top);
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 y =
          __floats2half2_rn(sgn * q[2 * e] * f.x, sgn * q[2 * e + 1] * f.x);
      u[e] = *reinterpret_cast<const uint32_t *>(&y);
    }
    const int64_t row = ((int64_t)h * p.N + tok) * p.G + (hq - h * p.G);
    *reinterpret_cast<uint4 *>(p.w.U + row * D + 8 * lane) = make_uint4(u[0], u[1], u[2], u[3]);
    if (lane == 0)
      p.w.rs[row] = fmaxf((float)(1.4426950408889634074 / KEY_FACTOR) * fabsf(p.scale) * f.y,
                          MIN_SCALE);
  }
}

template <int D>
struct Cfg {
  static constexpr int DB = D / 64;                // boxes of a Q, K or V tile
  static constexpr int TILE = DB * BOX;
  static constexpr int SK = 2, SV = 3;             // K and V stages
  static constexpr int OFF_K = HALVES * TILE;
  static constexpr int OFF_V = OFF_K + SK * TILE;
  static constexpr int OFF_ROW = OFF_V + SV * TILE;  // a word per row
  static constexpr int OFF_BAR = OFF_ROW + HALVES * BM * 4;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;  // + align slack
  // tensor memory columns: the halves' scores (their weights over them), then
  // their accumulators
  static constexpr int TMEM = 512, COL_O = HALVES * BN;
  static_assert(COL_O + HALVES * D <= TMEM, "tensor memory");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// V operand: keys along K in rows of 128 bytes (64 dims), 8-key groups 1024
// bytes apart (stride offset), 64-dim boxes `box` bytes apart (leading offset),
// 128-byte swizzle.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, uint32_t box) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(box >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// Pairs of fp32 in one register pair, one instruction for both.
using f32x2 = uint64_t;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves_of(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of a pair on the multiply-add pipe, for the share of the weights that
// the exponential unit has no time for.  x = n + f with n the nearest whole
// number, 2^f by the cubic with the least largest relative error on
// [-1/2, 1/2] (Remez exchange; 7.5e-5 = 2^-13.7, a fiftieth of the rounding to
// bf16 that follows), n added to the exponent.  x below -126 gives 2^-126, and
// so does a NaN: a row with one is made NaN through its maximum.
__device__ __forceinline__ float2 exp2_poly(f32x2 x) {
  constexpr float BIG = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  const float2 c = halves_of(x);
  x = pair(fmaxf(c.x, -126.f), fmaxf(c.y, -126.f));
  const f32x2 t = add2(x, pair(BIG, BIG));
  const f32x2 n = add2(t, pair(-BIG, -BIG));
  const f32x2 f = fma2(n, pair(-1.f, -1.f), x);
  f32x2 y = fma2(f, pair(0.0551716685f, 0.0551716685f), pair(0.2426111251f, 0.2426111251f));
  y = fma2(y, f, pair(0.6932609677f, 0.6932609677f));
  y = fma2(y, f, pair(0.9999280572f, 0.9999280572f));
  const float2 k = halves_of(t), v = halves_of(y);
  return make_float2(__uint_as_float(__float_as_uint(k.x) * 0x800000u + __float_as_uint(v.x)),
                     __uint_as_float(__float_as_uint(k.y) * 0x800000u + __float_as_uint(v.y)));
}

// Largest of the 64 scores at tS, NaN if one of them is; those from column lim
// on do not count.
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t tS, int lim) {
  uint32_t v[2][32];
#pragma unroll
  for (int c = 0; c < 2; ++c) ld32(tS + 32 * c, v[c]);
#pragma unroll
  for (int c = 0; c < 2; ++c) ld_wait(v[c]);
  float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float x = __uint_as_float(v[c][e]), y = __uint_as_float(v[c][e + 1]);
      if (MASK && 32 * c + e >= lim) x = -INFINITY;
      if (MASK && 32 * c + e + 1 >= lim) y = -INFINITY;
      t[(e >> 1) & 3] = max_nan(t[(e >> 1) & 3], max_nan(x, y));
    }
  return max_nan(max_nan(t[0], t[1]), max_nan(t[2], t[3]));
}

// Weights 2^(score rs + mm) of those 64, as bf16 over the first half of their
// columns, 32 scores at a time (each group's weights go where scores that have
// been read lay); returns the sum of the rounded weights.
template <bool MASK>
__device__ __forceinline__ float row_weights(uint32_t tS, int lim, float rs, float mm) {
  const f32x2 rs2 = pair(rs, rs), mm2 = pair(mm, mm);
  f32x2 sum[2] = {0, 0};
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t v[32], w[16];
    ld32(tS + 32 * c, v);
    ld_wait(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a = __uint_as_float(v[2 * e]), b = __uint_as_float(v[2 * e + 1]);
      if (MASK && 32 * c + 2 * e >= lim) a = -INFINITY;
      if (MASK && 32 * c + 2 * e + 1 >= lim) b = -INFINITY;
      const f32x2 x = fma2(pair(a, b), rs2, mm2);
      float2 y;
      if (!MASK && e % POLY_EVERY == POLY_EVERY - 1) {
        y = exp2_poly(x);
      } else {
        y = halves_of(x);
        y.x = fast_exp2(y.x);
        y.y = fast_exp2(y.y);
      }
      w[e] = pack_bf16x2(y.x, y.y);
      sum[e & 1] = add2(sum[e & 1], pair(__uint_as_float(w[e] << 16),
                                         __uint_as_float(w[e] & 0xffff0000u)));
    }
    st16(tS + 16 * c, w);
  }
  st_wait();
  const float2 s = halves_of(add2(sum[0], sum[1]));
  return s.x + s.y;
}

// N floats `step` apart, all on their way before the first is needed (volatile
// loads keep their order and are not sunk to their uses).
template <int N>
__device__ __forceinline__ void load_column(const float *q, int step, float *x) {
#pragma unroll
  for (int e = 0; e < N; ++e)
    asm volatile("ld.global.cg.f32 %0, [%1];\n" : "=f"(x[e]) : "l"(q + (int64_t)e * step));
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap map_u,
                  const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const Params p) {
  using C = Cfg<D>;
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
  const uint32_t kfull = bars(C::SK), kempty = bars(C::SK), vfull = bars(C::SV),
                 vempty = bars(C::SV), sfull = bars(HALVES), pready = bars(2 * HALVES),
                 ofree = bars(HALVES), pvdone = bars(2 * HALVES), ufull = bars(1),
                 uempty = bars(1), fin = bars(1);
  // two barriers a half for the value products in turn: whoever waits for a
  // tile's knows that the tile two before it is done, not the one before
  auto pv_bar = [&](int a, uint32_t t) { return pvdone + 16 * a + 8 * (t & 1u); };
  auto pv_phase = [](uint32_t t) { return (t >> 1) & 1u; };
  uint32_t *holder = reinterpret_cast<uint32_t *>(g + C::OFF_BAR + 496);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(g + C::OFF_BAR + 500);
  volatile int *join_flag = reinterpret_cast<volatile int *>(g + C::OFF_BAR + 504);  // per half
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::SK; ++i) {
      mbar_init(kfull + 8 * i, 1);
      mbar_init(kempty + 8 * i, 1);
    }
    for (int i = 0; i < C::SV; ++i) {
      mbar_init(vfull + 8 * i, 1);
      mbar_init(vempty + 8 * i, 1);
    }
    for (int a = 0; a < HALVES; ++a) {
      mbar_init(sfull + 8 * a, 1);
      mbar_init(pready + 16 * a, SM_WARPS / 2);
      mbar_init(pready + 16 * a + 8, SM_WARPS / 2);
      mbar_init(ofree + 8 * a, SM_WARPS);
      mbar_init(pvdone + 16 * a, 1);
      mbar_init(pvdone + 16 * a + 8, 1);
    }
    mbar_init(ufull, 1);
    mbar_init(uempty, 1);
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
  griddep_wait();  // the plan, the queries and the keys

  Seg s;
  bool more = seg_first(s, p);
  // halves of the segment's row tile that hold a row
  auto halves = [&]() { return (int64_t)s.n * p.G - (int64_t)s.mt * ROWS > BM ? 2 : 1; };

  if (warp < MMA_WARP) {
    // ---------------- softmax: thread = row r of half a, keys 64 c .. of a tile
    const int a = warp / SM_WARPS, c = (warp >> 2) & 1;
    const int r = 32 * (warp & 3) + lane;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t tS = trow + (uint32_t)(a * BN), tO = trow + (uint32_t)(C::COL_O + a * D);
    // The two warps of the same rows meet at a barrier of their own once a
    // tile.  A wait that ran out leaves by way of these meetings: nobody waits
    // at a barrier for a warp that has gone.
    const int pair_bar = 1 + 4 * a + (warp & 3), half_bar = 9 + a;
    auto any = [](int bar, int threads, bool x) {
      uint32_t y;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %3, 0;\n"
          " bar.red.or.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(y)
          : "r"(bar), "r"(threads), "r"((uint32_t)x)
          : "memory");
      __syncwarp();
      return y != 0;
    };
    // a word of the row's two threads: c = 1 leaves its part there, c = 0 what
    // both then go by
    volatile float *word = reinterpret_cast<volatile float *>(g + C::OFF_ROW) + a * BM + r;
    uint32_t it = 0, vt = 0;  // key tiles of this half so far; of the block
    bool ok = true;
    for (; more; more = seg_next(s, p)) {
      if (a >= halves()) {
        vt += s.nk;
        continue;
      }
      const int64_t row = (int64_t)s.mt * ROWS + a * BM + r;  // of the (sequence, KV head)
      const bool live = row < (int64_t)s.n * p.G &&
                        JL_IN_RANGE(p.err, s.start + row / p.G, 1, p.N);
      const bool any_live = row - lane < (int64_t)s.n * p.G;  // in this warp, and its partner
      const int tok = live ? (int)(row / p.G) : 0;
      const int seen = live ? min(s.L, max(0, s.L - s.n + tok + 1)) : 0;
      const int64_t urow = ((int64_t)s.h * p.N + s.start) * p.G + row;
      const float rs = live ? __ldcg(p.w.rs + urow) : 0.f;
      float m = 0.f, l = 0.f;
      for (int k = 0; k < s.nk; ++k, ++it, ++vt) {
        ok = wait_phase(sfull + 8 * a, it & 1u, abort_flag, p.err);
        __syncwarp();
        fence_after();
        const int t0 = (s.k0 + k) * BN;
        // values of keys past the last one, whatever their page holds there,
        // must not meet a weight of zero
        const int left = s.L - t0;
        if (a == 0 && c == 0 && left < BN) {
          const int vs = vt % C::SV;
          if (ok) ok = wait_phase(vfull + 8 * vs, (vt / C::SV) & 1u, abort_flag, p.err);
          uint8_t *V = g + C::OFF_V + vs * C::TILE + value_offset(r, p, D);
          if (ok && r >= left)
            for (int x = 0; x < C::DB; ++x)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4 *>(V + x * p.gran * 128 + 16 * e) =
                    make_uint4(0, 0, 0, 0);
          fence_async_smem();
        }
        const int lim = seen - t0;  // columns the row sees
        const bool all = __all_sync(~0u, lim >= BN);
        const int lim_c = lim - 64 * c;
        const uint32_t tC = tS + 64 * c;
        float top = -INFINITY;  // of the exponents
        if (any_live) {
          const float x = all ? row_max<false>(tC, BN) : row_max<true>(tC, lim_c);
          top = x == -INFINITY ? x : fmaf(x, rs, -m);
        }
        // both warps of the rows agree whether they need a new maximum
        const bool begin = k == 0;
        if (any(pair_bar, 64, begin || !(top <= RENEW) || !ok)) {
          if (c == 1) *word = top;
          if (any(pair_bar, 64, !ok)) {
            ok = false;
            break;
          }
          if (c == 0) {
            top = max_nan(top, *word);
            // a row that sees a NaN or an infinite score, or none that is finite,
            // is NaN from here on, whichever of its weights would show it
            if (top == INFINITY || (begin && lim > 0 && top == -INFINITY)) top = NAN;
            // (a row without a key so far refers to 0)
            *word = begin ? (top == -INFINITY ? 0.f : top) : top <= RENEW ? 0.f : top;
          }
          any(pair_bar, 64, false);
          const float up = *word;
          m += up;
          if (!begin) {
            // earlier products must have landed before the accumulator is scaled
            ok = wait_phase(pv_bar(a, it - 1), pv_phase(it - 1), abort_flag, p.err);
            __syncwarp();
            fence_after();
            const float f = up == 0.f ? 1.f : fast_exp2(-up);
            l *= f;
#pragma unroll 1
            for (int e0 = c * (D / 2); e0 < (c + 1) * (D / 2); e0 += 16) {
              uint32_t o[16];
              ld16(tO + e0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              st16(tO + e0, o);
            }
            st_wait();
            fence_before();
          }
          // (also: the words are free again)
          if (any(pair_bar, 64, !ok)) {
            ok = false;
            break;
          }
        }
        if (any_live)
          l += all ? row_weights<false>(tC, BN, rs, -m) : row_weights<true>(tC, lim_c, rs, -m);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready + 16 * a + 8 * c);
      }
      if (ok && s.nk > 0) {
        ok = wait_phase(pv_bar(a, it - 1), pv_phase(it - 1), abort_flag, p.err);
        __syncwarp();
        fence_after();
      }
      if (c == 1) *word = l;
      if (any(half_bar, SM_WARPS * 32, !ok)) break;
      if (c == 0) *word = l += *word;
      any(pair_bar, 64, false);
      l = *word;
      // output: the row itself, or its state where the row tile is split; each
      // warp the half of the dims that begins at d0
      const int d0 = c * (D / 2);
      const bool whole = s.k0 == 0 && s.k1 == s.units;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      uint16_t *out = p.out + ((int64_t)(s.start + tok) * p.Hq + s.h * p.G +
                               (row - (int64_t)tok * p.G)) * D;
      auto write_out = [&](int d, const uint32_t (&o)[16], float inv) {  // 16 dims from d on
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 q;
          uint32_t *qq = reinterpret_cast<uint32_t *>(&q);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float y = __uint_as_float(o[8 * e + 2 * x]),
                        z = __uint_as_float(o[8 * e + 2 * x + 1]);
            qq[x] = inv == 0.f ? 0u : pack_bf16x2(y * inv, z * inv);
          }
          *reinterpret_cast<uint4 *>(out + d + 8 * e) = q;
        }
      };
      // states of a split row tile: [half][d + 2][128 rows], a row per lane
      const Split split(s, p);
      constexpr int HALF = (D + 2) * BM;
      const int64_t mine = (split.record(blockIdx.x) * HALVES + a) * HALF + r;
      const bool mine_ok = JL_IN_RANGE(p.err, split.record(blockIdx.x), 1, 2 * SM_COUNT);
#pragma unroll 1
      for (int d = d0; d < d0 + D / 2; d += 16) {
        uint32_t o[16];
        if (s.nk > 0) {
          ld16(tO + d, o);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
        if (whole) {
          if (live) write_out(d, o, inv);
        } else if (mine_ok && any_live) {
#pragma unroll
          for (int e = 0; e < 16; ++e) p.w.part[mine + (d + e) * BM] = __uint_as_float(o[e]);
        }
      }
      if (s.nk > 0) {
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree + 8 * a);
      }
      if (!whole) {
        if (c == 0 && mine_ok) {
          p.w.part[mine + D * BM] = m;
          p.w.part[mine + (D + 1) * BM] = l;
        }
        // (the join is bound by what one SM gets from L2: 0.8 us per state of 256 rows)
        if (last_to_arrive(split, p, a, half_bar, SM_WARPS * 32, c == 0 && r == 0,
                           join_flag + a) && any_live) {
          auto record = [&](int64_t b) {
            return p.w.part + (split.record(b) * HALVES + a) * HALF + r;
          };
          float mj = -INFINITY, lj = 0.f;
          constexpr int M_AT_ONCE = 4, O_AT_ONCE = 2;  // records whose loads go side by side
#pragma unroll 1
          for (int64_t b = split.c0; b <= split.c1; b += M_AT_ONCE) {
            float x[M_AT_ONCE][2];
#pragma unroll
            for (int i = 0; i < M_AT_ONCE; ++i)
              load_column<2>(record(b + i < split.c1 ? b + i : split.c1) + D * BM, BM, x[i]);
#pragma unroll
            for (int i = 0; i < M_AT_ONCE; ++i) {
              const float mc = x[i][0], lc = x[i][1];
              if (b + i > split.c1 || lc == 0.f) continue;
              const float mn = fmaxf(mj, mc);
              lj = lj * (mj == mn ? 1.f : fast_exp2(mj - mn)) + lc * fast_exp2(mc - mn);
              mj = mn;
            }
          }
          const float ij = lj > 0.f || lj != lj ? 1.f / lj : 0.f;
#pragma unroll 1
          for (int d = d0; d < d0 + D / 2; d += 16) {
            float o[16] = {};
#pragma unroll 1
            for (int64_t b = split.c0; b <= split.c1; b += O_AT_ONCE) {
              float x[O_AT_ONCE][18];
#pragma unroll
              for (int i = 0; i < O_AT_ONCE; ++i) {
                const float *q = record(b + i < split.c1 ? b + i : split.c1);
                load_column<16>(q + d * BM, BM, x[i]);
                load_column<2>(q + D * BM, BM, x[i] + 16);
              }
#pragma unroll
              for (int i = 0; i < O_AT_ONCE; ++i) {
                const bool some = b + i <= split.c1 && x[i][17] != 0.f;
                const float w = some ? fast_exp2(x[i][16] - mj) : 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = some ? fmaf(w, x[i][e], o[e]) : o[e];
              }
            }
            if (live) {
              uint32_t ob[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e]);
              write_out(d, ob, ij);
            }
          }
        }
      }
      // the words are read before the next row tile's
      asm volatile("bar.sync %0, %1;\n" ::"r"(half_bar), "n"(SM_WARPS * 32) : "memory");
    }
  } else if (warp == MMA_WARP) {
    // ---------------- MMA issue: the halves in turn, values of a tile and then
    // the scores of the next
    constexpr uint32_t id_s = idesc_f16(BM, BN, 0);
    constexpr uint32_t id_o = idesc_f16(BM, D, 1) | (1u << 16);  // V along its N side
    const uint64_t du0 = desc_sw128(base), dk0 = desc_sw128(base + C::OFF_K);
    const uint64_t dv0 = desc_v(base + C::OFF_V, p.gran * 128);
    uint32_t voff[BN / 16];  // of 16 keys each, in descriptor units
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk) voff[kk] = value_offset(16 * kk, p, D) >> 4;
    bool ok = true;
    uint32_t kt = 0, sg = 0;            // key tiles and segments of the block
    uint32_t it0 = 0, it1 = 0, sg1 = 0; // key tiles of each half, segments of half 1
    auto wait_copy = [&](uint32_t bar, uint32_t ph) {
      return (bool)__all_sync(~0u, wait_phase(bar, ph, abort_flag, p.err));
    };
    auto wait = [&](uint32_t bar, uint32_t ph) {
      const bool w = wait_copy(bar, ph);
      fence_after();
      return w;
    };
    // half a, tile t of the block, tile it of the half: over the weights of the
    // tile before it
    auto scores = [&](int a, uint32_t t, uint32_t it) {
      if (it > 0 && !wait(pv_bar(a, it - 1), pv_phase(it - 1))) return false;
      if (elect_one()) {
        const uint64_t dk = dk0 + (uint64_t)(((t % C::SK) * C::TILE) >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = (uint32_t)(((i >> 2) * BOX + (i & 3) * 32) >> 4);
          mma_ss(tmem + a * BN, du0 + (uint64_t)((a * C::TILE) >> 4) + o, dk + o, id_s,
                 i ? 1u : 0u);
        }
        commit(sfull + 8 * a);
      }
      __syncwarp();
      return true;
    };
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      const int na = halves();
      if (!(ok = wait_copy(ufull, sg & 1u))) break;
      if (!(ok = wait_copy(kfull + 8 * (kt % C::SK), (kt / C::SK) & 1u))) break;
      for (int a = 0; ok && a < na; ++a) ok = scores(a, kt, a ? it1 : it0);
      if (!ok) break;
      if (elect_one()) commit(kempty + 8 * (kt % C::SK));
      __syncwarp();
      for (int k = 0; ok && k < s.nk; ++k, ++kt) {
        const uint32_t vs = kt % C::SV, nx = (kt + 1) % C::SK;
        for (int a = 0; a < na; ++a) {
          const uint32_t it = a ? it1 : it0, sa = a ? sg1 : sg;
          if (a == 0 && !(ok = wait_copy(vfull + 8 * vs, (kt / C::SV) & 1u))) break;
          if (k == 0 && sa > 0 && !(ok = wait(ofree + 8 * a, (sa - 1) & 1u))) break;
          const uint64_t dv = dv0 + (uint64_t)((vs * C::TILE) >> 4);
          for (int half = 0; half < 2; ++half) {  // of the tile's keys
            if (!(ok = wait(pready + 16 * a + 8 * half, it & 1u))) break;
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < BN / 32; ++i) {
                const int kk = half * (BN / 32) + i;
                mma_ts(tmem + C::COL_O + a * D, tmem + a * BN + 64 * half + 8 * i,
                       dv + voff[kk], id_o,
                       (k > 0 || kk > 0) ? 1u : 0u);
              }
              if (half) {
                commit(pv_bar(a, it));
                if (a == na - 1) commit(vempty + 8 * vs);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (k + 1 < s.nk) {
            if (a == 0 && !(ok = wait_copy(kfull + 8 * nx, ((kt + 1) / C::SK) & 1u))) break;
            if (!(ok = scores(a, kt + 1, it + 1))) break;
            if (a == na - 1) {
              if (elect_one()) commit(kempty + 8 * nx);
              __syncwarp();
            }
          }
          if (a) ++it1; else ++it0;
        }
      }
      if (elect_one()) commit(uempty);  // the queries have been read
      __syncwarp();
      ++sg;
      if (na > 1) ++sg1;
    }
    // every product has landed before the tensor memory is given back
    if (elect_one()) commit(fin);
    __syncwarp();
    drain_wait(fin, 0);
  } else {
    // ---------------- copies: queries of a segment, K and V of each key tile
    bool ok = true;
    uint32_t kt = 0, sg = 0;
    for (; ok && more; more = seg_next(s, p)) {
      if (s.nk == 0) continue;
      if (sg > 0 && !__all_sync(~0u, wait_phase(uempty, (sg - 1) & 1u, abort_flag, p.err))) break;
      const int na = halves();
      if (lane == 0) {
        mbar_expect_tx(ufull, na * C::TILE);
        const int64_t urow = ((int64_t)s.h * p.N + s.start) * p.G + (int64_t)s.mt * ROWS;
        for (int a = 0; a < na; ++a)
          for (int x = 0; x < C::DB; ++x)
            tma_load_2d(base + a * C::TILE + x * BOX, &map_u, x * 64, (int)urow + a * BM, ufull);
      }
      __syncwarp();
      ++sg;
      // lane i copies granule i of V; the next tile's page is looked up meanwhile
      auto place = [&](int k, bool &here) -> int64_t {
        const int t = (s.k0 + k) * BN + p.gran * lane;
        here = k < s.nk && lane < BN >> p.gran_log && t < s.L;
        return here ? ((int64_t)page_of(p, s.b, t) * p.Hkv + s.h) * p.P + t % p.P : 0;
      };
      bool here;
      int64_t row = place(0, here);
      const int64_t krow = ((int64_t)s.b * p.Hkv + s.h) * p.key_tiles;
      for (int k = 0; k < s.nk; ++k) {
        const int ks = kt % C::SK, vs = kt % C::SV;
        if (!__all_sync(~0u, wait_phase(kempty + 8 * ks, ((kt / C::SK) & 1u) ^ 1u, abort_flag,
                                        p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_expect_tx(kfull + 8 * ks, C::TILE);
          for (int x = 0; x < C::DB; ++x)
            tma_load_2d(base + C::OFF_K + ks * C::TILE + x * BOX, &map_k, x * 64,
                        (int)((krow + s.k0 + k) * BN), kfull + 8 * ks);
        }
        __syncwarp();
        const int grans = __popc(__ballot_sync(~0u, here));
        const bool vok = __all_sync(
            ~0u, wait_phase(vempty + 8 * vs, ((kt / C::SV) & 1u) ^ 1u, abort_flag, p.err));
        ++kt;  // this tile's keys are on their way
        if (!vok) {
          ok = false;
          break;
        }
        const uint32_t bytes = p.gran * D * 2;
        if (lane == 0) mbar_expect_tx(vfull + 8 * vs, grans * bytes);
        __syncwarp();
        if (here)
          tma_load_3d(base + C::OFF_V + vs * C::TILE + lane * bytes, &map_v, 0, (int)row, 0,
                      vfull + 8 * vs);
        __syncwarp();
        row = place(k + 1, here);
      }
    }
    if (*abort_flag) {  // let the copies in flight land before the block leaves
      if (sg > 0) drain_wait(ufull, (sg - 1) & 1u);
      for (uint32_t i = kt > C::SK ? kt - C::SK : 0; i < kt; ++i)
        drain_wait(kfull + 8 * (i % C::SK), (i / C::SK) & 1u);
      const uint32_t vt = ok || kt == 0 ? kt : kt - 1;  // the last tile's V may not have left
      for (uint32_t i = vt > C::SV ? vt - C::SV : 0; i < vt; ++i)
        drain_wait(vfull + 8 * (i % C::SV), (i / C::SV) & 1u);
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

template <int D>
cudaError_t launch_many_t(const Params &p, const ChunkArgs &a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap map_u, map_k, map_v;
  const int64_t rows = p.N * p.Hq;
  if (!tc::make_map(&map_u, p.w.U, rows, D, D, BM) ||
      !tc::make_map(&map_k, p.w.keys, (uint64_t)p.B * p.Hkv * p.key_tiles * BN, D, D, BN) ||
      !make_value_map(&map_v, a.value_pages, (uint64_t)p.num_pages * p.Hkv * p.P, D, p.gran))
    return cudaErrorInvalidValue;
  const int64_t blocks = (rows + PREP_THREADS / (D / 8) - 1) / (PREP_THREADS / (D / 8));
  const int64_t most = (int64_t)p.blocks * 8;
  const uint64_t al = (uint64_t)reinterpret_cast<uintptr_t>(p.Q) |
                      (uint64_t)(p.q_tok | p.q_head) * (a.q_f32 ? 4 : 2);
  const bool vec = (al & 15) == 0;
  auto prep = a.q_f32 ? (vec ? prep_kernel<D, true, true> : prep_kernel<D, true, false>)
                      : (vec ? prep_kernel<D, false, true> : prep_kernel<D, false, false>);
  prep<<<(unsigned)(1 + (blocks < most ? blocks : most)), PREP_THREADS, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_expand_paged(p.codes, p.norms, p.num_pages, p.P, p.table, p.max_pages, p.lens, p.B,
                          p.Hkv, p.max_len, p.S, a.m, D, p.w.keys, stream);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_after(attend_kernel<D>, p.blocks, THREADS, C::SMEM, stream, map_u, map_k, map_v, p);
}

}  // namespace

size_t many_workspace(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int d, Work *w,
                      void *base) {
  return lay_out(w, base, N, B, Hq, Hkv, ROWS, d, (size_t)ROWS * (d + 2),
                 (size_t)B * Hkv * ((max_len + BN - 1) / BN) * BN * d * 2);
}

cudaError_t launch_many(Params p, const ChunkArgs &a, cudaStream_t stream) {
  p.rows = ROWS;
  many_workspace(p.N, p.B, p.Hq, p.Hkv, p.max_len, a.d, &p.w, a.workspace);
  return a.d == 128 ? launch_many_t<128>(p, a, stream) : launch_many_t<64>(p, a, stream);
}

}  // namespace chunk
}  // namespace jlk
