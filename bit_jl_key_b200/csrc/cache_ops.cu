// cache_ops.cu -- what a serving loop does to a paged compressed cache between
// attention calls: store a chunk of coded keys, accumulate the attention
// weight each key received, and evict the keys that received the least.
//
//   store   key i of sequence b goes to position seq_lens[b] + i, that is to
//           page block_table[b][pos / P], slot pos % P.  A copy.
//   weight  mass'[b][kv][t] = decay mass[b][kv][t]
//                             + sum over the KV head's query heads of softmax_t(scale s[t]).
//   evict   of the L keys of a (sequence, KV head), the first `sink`, the last
//           `recent`, and of the others the ones with the largest mass (equal
//           masses: the lower index) up to `keep` in all, in their order.
//
// All three are bound by memory, small calls by the latency of a launch; the
// selection of the eviction is a radix select whose histograms and prefix sums
// are shared by a cluster of blocks.
#include "jl_common.cuh"
#include "jl_internal.h"

#include <cooperative_groups.h>

namespace jlk {

namespace cg = cooperative_groups;

namespace {

// The pools of a paged cache, as bytes are moved: a key's code is W words, its
// norms c binary16s, its value d bf16s.
struct Pools {
  uint32_t *codes;
  uint16_t *norms, *values;
  int num_pages, P, Hkv, W, c, d;
  int *err;
  __device__ __forceinline__ int64_t rows() const { return (int64_t)num_pages * Hkv * P; }
};

__device__ __forceinline__ int64_t pool_row(const Pools &p, int page, int head, int slot) {
  return ((int64_t)page * p.Hkv + head) * p.P + slot;
}

// Page of position pos, or -1 (recorded) where the table has no such column
// or names a page outside the pool.
__device__ __forceinline__ int table_page(const int32_t *table, int max_pages, int b, int64_t pos,
                                          const Pools &p) {
  const int64_t col = pos / p.P;
  int page = -1;
  if (pos >= 0 && col < max_pages) page = __ldg(table + (int64_t)b * max_pages + col);
  if (page < 0 || page >= p.num_pages) {
    record_device_error(p.err, DERR_PAGE);
    return -1;
  }
  return page;
}

// Moves the keys of a warp: lane i names one (its row among the sources, its
// pool row; a negative pool row moves nothing), then d / 8 lanes move a key at
// a time, 16 bytes of its value each, UNROLL keys' loads in flight.  Where keys
// come from is `src`: value(row), code(row), norm(row) pointers.
constexpr int UNROLL = 4;
template <int D, int UNIT, typename Src>
__device__ __forceinline__ void move_keys(const Pools &p, const Src &src, int64_t from,
                                          int64_t to) {
  constexpr int LANES = D / 8, PER = 32 / LANES;  // lanes of a key, keys side by side
  const int lane = threadIdx.x & 31, g = lane / LANES, l = lane % LANES;
  const int units = p.W / UNIT;                   // of UNIT words of a code
#pragma unroll 1
  for (int i0 = 0; i0 < LANES; i0 += UNROLL) {
    int64_t f[UNROLL], t[UNROLL];
    uint4 v[UNROLL];
    uint32_t c[UNROLL][UNIT];
    uint16_t n[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int who = (i0 + i) * PER + g;
      f[i] = __shfl_sync(~0u, from, who);
      t[i] = __shfl_sync(~0u, to, who);
      if (!JL_IN_RANGE(p.err, t[i] < 0 ? 0 : t[i], 1, p.rows()) ||
          !JL_IN_RANGE(p.err, t[i] < 0 ? 0 : f[i], 1, src.rows()))
        t[i] = -1;
      if (t[i] < 0) continue;
      v[i] = *reinterpret_cast<const uint4 *>(src.value(f[i]) + 8 * l);
      if (l < units) {
        const uint32_t *w = src.code(f[i]) + l * UNIT;
        if constexpr (UNIT == 4) {
          const uint4 x = *reinterpret_cast<const uint4 *>(w);
          c[i][0] = x.x; c[i][1] = x.y; c[i][2] = x.z; c[i][3] = x.w;
        } else {
#pragma unroll
          for (int e = 0; e < UNIT; ++e) c[i][e] = w[e];
        }
      }
      if (l < p.c) n[i] = src.norm(f[i])[l];
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      if (t[i] < 0) continue;
      *reinterpret_cast<uint4 *>(p.values + t[i] * D + 8 * l) = v[i];
      if (l < units) {
        uint32_t *w = p.codes + t[i] * p.W + l * UNIT;
        if constexpr (UNIT == 4) {
          *reinterpret_cast<uint4 *>(w) = make_uint4(c[i][0], c[i][1], c[i][2], c[i][3]);
        } else {
#pragma unroll
          for (int e = 0; e < UNIT; ++e) w[e] = c[i][e];
        }
      }
      // codes of more units than a key has lanes
      for (int u = l + LANES; u < units; u += LANES)
        for (int e = 0; e < UNIT; ++e)
          p.codes[t[i] * p.W + u * UNIT + e] = src.code(f[i])[u * UNIT + e];
      if (l < p.c) p.norms[t[i] * p.c + l] = n[i];
    }
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// store

namespace store {

constexpr int THREADS = 128;

struct Params {
  Pools pool;
  const uint32_t *codes;  // [N][Hkv][W]
  const uint16_t *norms;  // [N][Hkv][c]
  const uint16_t *V;      // strided [N][Hkv][d]
  int64_t v_tok, v_head;
  const int32_t *cu, *table, *lens;
  int B, max_pages;
  int64_t N;
};

struct Chunk {
  const Params &p;
  int h;
  __device__ int64_t rows() const { return p.N; }
  __device__ const uint16_t *value(int64_t r) const { return p.V + r * p.v_tok + h * p.v_head; }
  __device__ const uint32_t *code(int64_t r) const {
    return p.codes + (r * p.pool.Hkv + h) * p.pool.W;
  }
  __device__ const uint16_t *norm(int64_t r) const {
    return p.norms + (r * p.pool.Hkv + h) * p.pool.c;
  }
};

// A warp takes 32 consecutive tokens of one KV head, whose rows are neighbours
// in a page; each lane finds its token's sequence and place.  Bound by memory:
// 16384 tokens x 8 heads of 308 bytes are 80.7 MB read and written in 15.5 us
// (5.2 TB/s; 18.6 us as called, 17.1 in a graph); 40 tokens take 7 us in a graph.
template <int D, int UNIT>
__global__ void __launch_bounds__(THREADS) store_kernel(const Params p) {
  const int h = blockIdx.y;
  const int64_t r = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  int64_t to = -1;
  // (rows outside every sequence are a batch's padding)
  if (r < p.N && r >= __ldg(p.cu) && r < __ldg(p.cu + p.B)) {
    int lo = 0, hi = p.B;  // the last b with cu[b] <= r
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) <= r) lo = mid; else hi = mid;
    }
    const int64_t pos = (int64_t)__ldg(p.lens + lo) + (r - __ldg(p.cu + lo));
    const int page = table_page(p.table, p.max_pages, lo, pos, p.pool);
    if (page >= 0) to = pool_row(p.pool, page, h, (int)(pos % p.pool.P));
  }
  move_keys<D, UNIT>(p.pool, Chunk{p, h}, r, to);
}

}  // namespace store

cudaError_t launch_store_paged(const StoreArgs &a, cudaStream_t stream) {
  store::Params p{};
  p.pool = {a.code_pages, a.norm_pages, a.value_pages, a.num_pages, a.page_tokens,
            a.Hkv, a.words, a.norms_per_key, a.d, device_error_ptr()};
  if (!p.pool.err) return cudaErrorInvalidSymbol;
  p.codes = a.codes; p.norms = a.norms; p.V = a.V;
  p.v_tok = a.v_tok; p.v_head = a.v_head;
  p.cu = a.cu_seqlens; p.table = a.block_table; p.lens = a.seq_lens;
  p.B = a.B; p.max_pages = a.max_pages; p.N = a.N;
  const dim3 grid((unsigned)((a.N + store::THREADS - 1) / store::THREADS), a.Hkv);
  // 16 bytes of a code at a time where the chunk's codes allow it (a pool's do)
  const bool four = a.words % 4 == 0 && (reinterpret_cast<uintptr_t>(a.codes) & 15) == 0;
  auto kernel = a.d == 128 ? (four ? store::store_kernel<128, 4> : store::store_kernel<128, 1>)
                           : (four ? store::store_kernel<64, 4> : store::store_kernel<64, 1>);
  kernel<<<grid, store::THREADS, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// accumulated attention weight

namespace mass {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int LOADS = 4;  // of a thread, in flight

struct Params {
  const float *scores;  // [B][Hq][T]
  const float *mass;    // [B][Hkv][T] (not read when decay is 0)
  float *out;
  const int32_t *lens;
  int Hq, Hkv, G;
  int64_t T;
  bool out_vec;          // out is 16-byte aligned
  // scores are read times `half`, softmax_scale's sign over 2, so that no
  // difference of two overflows; k, of such a difference: 2 |softmax_scale| log2(e)
  float k, half, decay;
  int *err;
};

struct MS {
  float m, l;
};
// Joins two softmax states; a state without keys is (-inf, 0), and one with a
// NaN among them NaN in both.  The maximum is of the scores themselves (times
// `half`): only differences are scaled, so a row of the type's lowest value is as
// uniform as any other.
__device__ __forceinline__ MS join(MS a, MS b, float k) {
  const float m = max_nan(a.m, b.m);
  if (m == -INFINITY) return {m, 0.f};
  return {m, a.l * exp2f((a.m - m) * k) + b.l * exp2f((b.m - m) * k)};
}

// VEC entries from place i on of the block's n, times `f`; -inf from n on.
template <int VEC>
__device__ __forceinline__ void load_scores(const float *s, int i, int n, float f,
                                            float (&x)[VEC]) {
  if (i + VEC <= n) {
    if constexpr (VEC == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(s + i);
      x[0] = v.x * f; x[1] = v.y * f; x[2] = v.z * f; x[3] = v.w * f;
    } else {
      x[0] = s[i] * f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = i + e < n ? s[i + e] * f : -INFINITY;
  }
}

// One cluster per (sequence, KV head); its blocks split the keys.  Pass one
// reads the scores of the group's heads, two at a time so that their loads are
// in flight together, for the softmax states, which the blocks exchange through
// distributed shared memory; pass two reads the scores again, from L2, and
// writes the weights.  (Keeping them in shared memory in between measured no
// faster: it costs resident blocks.)  8 sequences of up to 32768 keys, 32 over 8
// heads, are 40 MB in 22.4 us as called and 17.9 in a graph, where the bytes alone
// would take 6.3.  The rest is this form's latency: a first trip to memory in each
// of two passes and the blocks' two meetings between them, all for a maximum and a
// sum per head.  A caller that had those, as a decode step does inside, would need
// one pass.
template <int VEC>
__global__ void __launch_bounds__(THREADS) mass_kernel(const Params p) {
  extern __shared__ MS ms_smem[];            // [G][WARPS], then [G] of the block, [G] of all
  MS *part = ms_smem, *mine = ms_smem + p.G * WARPS, *all = mine + p.G;
  cg::cluster_group cl = cg::this_cluster();
  const int nb = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int unit = blockIdx.x / nb, b = unit / p.Hkv, h = unit - b * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t L = __ldg(p.lens + b);
  if (L < 0 || L > p.T) {
    if (threadIdx.x == 0) record_device_error(p.err, DERR_DECODE_PLAN);
    L = L < 0 ? 0 : p.T;
  }
  int64_t share = (L + nb - 1) / nb;
  share = (share + VEC - 1) / VEC * VEC;
  const int64_t t0 = rank * share < L ? rank * share : L;
  const int64_t t1 = t0 + share < L ? t0 + share : L;
  // (every access below is inside the block's n keys of its rows)
  const int n = JL_IN_RANGE(p.err, t0, t1 - t0, p.T) ? (int)(t1 - t0) : 0;
  const float *s0 = p.scores + ((int64_t)b * p.Hq + (int64_t)h * p.G) * p.T + t0;

  constexpr int STEP = THREADS * VEC;
  for (int g = 0; g < p.G; g += 2) {
    const float *s = s0 + (int64_t)g * p.T;
    const int64_t more = g + 1 < p.G ? p.T : 0;  // an odd head out is read twice
    MS a[2] = {{-INFINITY, 0.f}, {-INFINITY, 0.f}};
    for (int t = threadIdx.x * VEC; t < n; t += STEP * LOADS) {
      float x[2][LOADS][VEC];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
          load_scores<VEC>(s + i * more, t + q * STEP, n, p.half, x[i][q]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float m = a[i].m;
#pragma unroll
        for (int q = 0; q < LOADS; ++q)
#pragma unroll
          for (int e = 0; e < VEC; ++e) m = max_nan(m, x[i][q][e]);
        if (m != -INFINITY) {
          float l = a[i].l * fast_exp2((a[i].m - m) * p.k);
#pragma unroll
          for (int q = 0; q < LOADS; ++q)
#pragma unroll
            for (int e = 0; e < VEC; ++e) l += fast_exp2((x[i][q][e] - m) * p.k);
          a[i] = {m, l};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 16; o; o >>= 1)
        a[i] = join(a[i], {__shfl_xor_sync(~0u, a[i].m, o), __shfl_xor_sync(~0u, a[i].l, o)}, p.k);
      if (lane == 0 && g + i < p.G) part[(g + i) * WARPS + warp] = a[i];
    }
  }
  __syncthreads();
  // a warp joins a head's states, one of each of its lanes
  for (int g = warp; g < p.G; g += WARPS) {
    MS a = lane < WARPS ? part[g * WARPS + lane] : MS{-INFINITY, 0.f};
#pragma unroll
    for (int o = 16; o; o >>= 1)
      a = join(a, {__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.l, o)}, p.k);
    if (lane == 0) mine[g] = a;
  }
  // the older weights, on their way while the blocks meet
  const int64_t row = ((int64_t)b * p.Hkv + h) * p.T + t0;
  const int first = threadIdx.x * VEC;
  float old[2][VEC] = {};
  auto load_old = [&](int t) {
    if (p.decay != 0.f) {
#pragma unroll
      for (int q = 0; q < 2; ++q) load_scores<VEC>(p.mass + row, t + q * STEP, n, p.decay, old[q]);
    }
  };
  load_old(first);
  cl.sync();
  for (int g = threadIdx.x; g < p.G; g += THREADS) {
    MS a{-INFINITY, 0.f};
    MS x[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = r < nb ? cl.map_shared_rank(mine, r)[g] : a;
#pragma unroll
    for (int r = 0; r < 8; ++r) a = join(a, x[r], p.k);
    // weight = 2^((x - m) k - log2 l); a head whose keys are all -inf adds nothing
    all[g] = a.m == -INFINITY ? MS{0.f, -INFINITY} : MS{a.m, -log2f(a.l)};
  }
  cl.sync();  // also: no block leaves while another reads its states
  for (int t = first; t < n; t += STEP * 2) {
    if (t != first) load_old(t);
    float w[2][VEC] = {};
#pragma unroll 4
    for (int g = 0; g < p.G; ++g) {
      const MS a = all[g];
      float x[2][VEC];
#pragma unroll
      for (int q = 0; q < 2; ++q)
        load_scores<VEC>(s0 + (int64_t)g * p.T, t + q * STEP, n, p.half, x[q]);
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[q][e] += fast_exp2(fmaf(x[q][e] - a.m, p.k, a.l));
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int tq = t + q * STEP;
      float *o = p.out + row + tq;
      if (VEC == 4 && p.out_vec && tq + VEC <= n) {
        *reinterpret_cast<float4 *>(o) =
            make_float4(old[q][0] + w[q][0], old[q][1 % VEC] + w[q][1 % VEC],
                        old[q][2 % VEC] + w[q][2 % VEC], old[q][3 % VEC] + w[q][3 % VEC]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (tq + e < n) o[e] = old[q][e] + w[q][e];
      }
    }
  }
}

}  // namespace mass

namespace {
template <typename K, typename P>
cudaError_t launch_cluster(K kernel, int64_t blocks, int cluster, int threads, size_t smem,
                           cudaStream_t stream, const P &p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Blocks per (sequence, KV head): as many as give the device 256 of them, while
// each keeps `least` keys, up to the portable cluster size.  (Weights, 4 against 8
// blocks: 64 units of 32768 keys 20.5 and 28 us, 32 units of 131072 keys 29 and
// 19.5 us.  Selection, 64 units of 32768 keys: 41 and 55 us when this was chosen.)
int cluster_for(int64_t units, int64_t keys, int least) {
  int c = 1;
  while (c < 8 && units * c < 256 && keys / (2 * c) >= least) c *= 2;
  return c;
}
}  // namespace

cudaError_t launch_accumulate(const AccumulateArgs &a, cudaStream_t stream) {
  mass::Params p{};
  p.scores = a.scores; p.mass = a.mass; p.out = a.out; p.lens = a.seq_lens;
  p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.T = a.max_len;
  // (a scale of 0 stays above it, so that -inf times it is -inf: as the least
  // positive number, by which no difference comes to 2^-20; and none is infinite,
  // so that 0 times it is 0)
  p.k = fminf(fmaxf(fabsf(a.softmax_scale) * 2.88539008177792681472f, 1.40129846e-45f),
              3.40282347e+38f);
  p.half = a.softmax_scale < 0.f ? -0.5f : 0.5f;
  p.decay = a.decay;
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidSymbol;
  const int64_t units = (int64_t)a.B * a.Hkv;
  const int cluster = cluster_for(units, a.max_len, 1024);
  const size_t smem = (size_t)p.G * (mass::WARPS + 2) * sizeof(mass::MS);  // <= 72 KB: G <= 512
  auto al = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool vec = a.max_len % 4 == 0 && al(a.scores) && (a.decay == 0.f || al(a.mass));
  p.out_vec = al(a.out);
  auto kernel = vec ? mass::mass_kernel<4> : mass::mass_kernel<1>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, units * cluster, cluster, mass::THREADS, smem, stream, p);
}

// ---------------------------------------------------------------------------
// eviction

namespace evict {

constexpr int THREADS = 512, WARPS = THREADS / 32;
constexpr int BINS = 256, COPIES = 8;  // of a histogram: equal digits in a warp are common
constexpr int COPY_THREADS = EVICT_KEYS, MAX_CLUSTER = 8;

struct Params {
  Pools pool;
  const float *mass;  // [B][Hkv][T]
  const int32_t *lens, *src_table, *dst_table;
  int src_pages, dst_pages, B;
  int64_t T;
  int keep, recent, sink, cached;  // cached: the block's sort keys fit in shared memory
  int32_t *out_index, *out_lens;
  float *out_mass;
};

// Sort key: larger mass, larger key.  -0 equals +0; a NaN ranks below all.
__device__ __forceinline__ uint32_t sort_key(float x) {
  if (isnan(x)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int64_t sequence_length(const Params &p, int b) {
  int64_t L = __ldg(p.lens + b);
  if (L < 0 || L > p.T) {
    if (threadIdx.x == 0) record_device_error(p.pool.err, DERR_DECODE_PLAN);
    L = L < 0 ? 0 : p.T;
  }
  return L;
}

// Exclusive prefix of a pair of counts over the block; totals in (ta, tb).
__device__ __forceinline__ void block_scan(int &a, int &b, int &ta, int &tb, int2 *sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int xa = __shfl_up_sync(~0u, ia, o), xb = __shfl_up_sync(~0u, ib, o);
    if (lane >= o) { ia += xa; ib += xb; }
  }
  if (lane == 31) sh[warp] = make_int2(ia, ib);
  __syncthreads();
  if (warp == 0) {
    int2 v = lane < WARPS ? sh[lane] : make_int2(0, 0);
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
      const int xa = __shfl_up_sync(~0u, v.x, o), xb = __shfl_up_sync(~0u, v.y, o);
      if (lane >= o) { v.x += xa; v.y += xb; }
    }
    if (lane < WARPS) sh[lane] = v;
  }
  __syncthreads();
  const int2 before = warp ? sh[warp - 1] : make_int2(0, 0), tot = sh[WARPS - 1];
  a = before.x + ia - a;
  b = before.y + ib - b;
  ta = tot.x;
  tb = tot.y;
  __syncthreads();
}

// Word of a block's i-th sort key: one word in 33 is left out, so that threads
// that each read a run of neighbouring keys meet in no bank.
__host__ __device__ __forceinline__ int64_t place(int64_t i) { return i + (i >> 5); }

// Which keys stay.  A cluster per (sequence, KV head), whose blocks own
// neighbouring ranges of keys.  The `need` largest masses of the candidates
// (all but the first `sink` and the last `recent`) are those above the
// threshold key found 8 bits at a time from histograms summed over the
// cluster, and the first ones of those equal to it; a prefix sum over the
// blocks then numbers the kept keys in order.  Bound by latency: of 25 us in the
// kernel (64 units of 32768 keys) 4 go to the loads, 3.8 to each of the four
// digits (counting 1.5, the blocks' meeting 1.2, sum and search 1.1) and 6 to
// numbering and writing the indices.
__global__ void __launch_bounds__(THREADS) select_kernel(const Params p) {
  extern __shared__ uint32_t cache[];  // the block's sort keys, if they fit
  __shared__ uint32_t copies[BINS * COPIES], hist[2][BINS], sum[BINS];
  __shared__ int2 scan[WARPS];
  __shared__ int2 counts;              // of this block: kept for sure, equal to the threshold
  __shared__ uint32_t s_digit;
  __shared__ int s_above;
  cg::cluster_group cl = cg::this_cluster();
  const int nb = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int unit = blockIdx.x / nb, b = unit / p.pool.Hkv, h = unit - b * p.pool.Hkv;
  const int64_t L = sequence_length(p, b);
  const int64_t keep = L < p.keep ? L : p.keep;
  const float *m = p.mass + (int64_t)unit * p.T;
  int32_t *idx = p.out_index + (int64_t)unit * p.keep;
  if (rank == 0 && h == 0 && threadIdx.x == 0) p.out_lens[b] = (int32_t)keep;
  const int64_t stride = (int64_t)nb * THREADS, me = (int64_t)rank * THREADS + threadIdx.x;
  for (int64_t j = keep + me; j < p.keep; j += stride) idx[j] = -1;
  if (L <= p.keep) {  // every key stays (the same for the whole cluster)
    for (int64_t j = me; j < L; j += stride) idx[j] = (int32_t)j;
    return;
  }
  const int64_t share = (L + nb - 1) / nb;
  const int64_t t0 = rank * share < L ? rank * share : L;
  const int64_t t1 = t0 + share < L ? t0 + share : L;
  const int64_t c0 = p.sink, c1 = L - p.recent;  // candidates [c0, c1)
  if (p.cached) {
    constexpr int AT_ONCE = 8;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += THREADS * AT_ONCE) {
      float x[AT_ONCE];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
        if (t + q * THREADS < t1) x[q] = m[t + q * THREADS];
#pragma unroll
      for (int q = 0; q < AT_ONCE; ++q)
        if (t + q * THREADS < t1) cache[place(t + q * THREADS - t0)] = sort_key(x[q]);
    }
    __syncthreads();
  }
  auto key = [&](int64_t t) { return p.cached ? cache[place(t - t0)] : sort_key(m[t]); };

  int need = (int)(keep - p.sink - p.recent);    // of the candidates; may be 0
  uint32_t prefix = 0, mask = 0;                 // threshold digits found so far
  for (int i = threadIdx.x; i < BINS * COPIES; i += THREADS) copies[i] = 0;
  __syncthreads();
  for (int shift = 24; shift >= 0; shift -= 8) {
    const int64_t a = t0 > c0 ? t0 : c0, z = t1 < c1 ? t1 : c1;
    for (int64_t t = a + threadIdx.x; t < z; t += THREADS) {
      const uint32_t k = key(t);
      if ((k & mask) == prefix)
        atomicAdd(&copies[((k >> shift) & 255u) * COPIES + (threadIdx.x & (COPIES - 1))], 1u);
    }
    __syncthreads();
    // two histograms in turn: a block still reading one may not see it change
    uint32_t *mine = hist[(shift >> 3) & 1];
    for (int i = threadIdx.x; i < BINS; i += THREADS) {
      uint32_t v = 0;
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        v += copies[i * COPIES + c];
        copies[i * COPIES + c] = 0;
      }
      mine[i] = v;
    }
    cl.sync();
    for (int i = threadIdx.x; i < BINS; i += THREADS) {
      uint32_t v = 0;
#pragma unroll
      for (int r = 0; r < MAX_CLUSTER; ++r)
        if (r < nb) v += cl.map_shared_rank(mine, r)[i];
      sum[i] = v;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // the digit where the count from above first reaches need: lane i
      // holds bins 255 - 8 i downwards
      uint32_t v[8], tot = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) tot += v[e] = sum[255 - (8 * threadIdx.x + e)];
      uint32_t inc = tot;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(~0u, inc, o);
        if ((int)threadIdx.x >= o) inc += x;
      }
      uint32_t above = inc - tot;
      const bool here = above < (uint32_t)need && inc >= (uint32_t)need;
      if (here) {
        int e = 0;
        while (above + v[e] < (uint32_t)need) above += v[e++];
        s_digit = 255 - (8 * threadIdx.x + e);
        s_above = (int)above;
      }
      if (need == 0 && threadIdx.x == 0) {
        s_digit = 255;  // nothing is above the threshold, none of the equal is taken
        s_above = 0;
      }
    }
    __syncthreads();
    need -= s_above;
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    __syncthreads();
  }
  const uint32_t tau = prefix;  // keys above it stay, and the first `need` equal to it

  // A thread owns neighbouring keys, so that one prefix sum over the block and
  // the cluster numbers its kept keys: those that stay for sure, and of those
  // equal to tau the first `need`.
  auto classify = [&](int64_t t, int &sure, int &tie) {
    const uint32_t k = key(t);
    const bool held = t < c0 || t >= c1;
    sure = held || k > tau;
    tie = !held && k == tau;
  };
  const int64_t own = (share + THREADS - 1) / THREADS;
  const int64_t a0 = t0 + threadIdx.x * own < t1 ? t0 + threadIdx.x * own : t1;
  const int64_t a1 = a0 + own < t1 ? a0 + own : t1;
  int na = 0, nt = 0, ta, tb;
  for (int64_t t = a0; t < a1; ++t) {
    int s, e;
    classify(t, s, e);
    na += s;
    nt += e;
  }
  block_scan(na, nt, ta, tb, scan);
  if (threadIdx.x == 0) counts = make_int2(ta, tb);
  cl.sync();
#pragma unroll
  for (int r = 0; r < MAX_CLUSTER; ++r)
    if (r < rank) {
      const int2 v = *cl.map_shared_rank(&counts, r);
      na += v.x;
      nt += v.y;
    }
  for (int64_t t = a0; t < a1; ++t) {
    int s, e;
    classify(t, s, e);
    const int j = na + (nt < need ? nt : need);
    if ((s || (e && nt < need)) && JL_IN_RANGE(p.pool.err, j, 1, keep)) idx[j] = (int32_t)t;
    na += s;
    nt += e;
  }
  cl.sync();  // no block leaves while another reads its counts
}

struct Cache {
  const Pools &p;
  __device__ int64_t rows() const { return p.rows(); }
  __device__ const uint16_t *value(int64_t r) const { return p.values + r * p.d; }
  __device__ const uint32_t *code(int64_t r) const { return p.codes + r * p.W; }
  __device__ const uint16_t *norm(int64_t r) const { return p.norms + r * p.c; }
};

// Moves the kept keys, 32 neighbouring slots of the new pages to a warp.  Bound by
// memory: 1.05 M keys of 290 bytes, 0.61 GB read and written, in 111 us (5.5 TB/s).
template <int D, int UNIT>
__global__ void __launch_bounds__(COPY_THREADS) move_kernel(const Params p) {
  griddep_wait();
  const int tiles = (int)evict_blocks(p.keep);
  const int unit = blockIdx.x / tiles, b = unit / p.pool.Hkv, h = unit - b * p.pool.Hkv;
  const int64_t j = (int64_t)(blockIdx.x - unit * tiles) * COPY_THREADS + threadIdx.x;
  int64_t from = 0, to = -1;
  const int t = j < p.keep ? __ldcg(p.out_index + (int64_t)unit * p.keep + j) : -1;
  if (j < p.keep && JL_IN_RANGE(p.pool.err, t < 0 ? 0 : t, 1, p.T))
    p.out_mass[(int64_t)unit * p.keep + j] = t >= 0 ? p.mass[(int64_t)unit * p.T + t] : 0.f;
  if (t >= 0) {
    const int sp = table_page(p.src_table, p.src_pages, b, t, p.pool);
    const int dp = table_page(p.dst_table, p.dst_pages, b, j, p.pool);
    if (sp >= 0 && dp >= 0) {
      from = pool_row(p.pool, sp, h, t % p.pool.P);
      to = pool_row(p.pool, dp, h, (int)(j % p.pool.P));
    }
  }
  move_keys<D, UNIT>(p.pool, Cache{p.pool}, from, to);
}

}  // namespace evict

cudaError_t launch_evict_paged(const EvictArgs &a, cudaStream_t stream) {
  evict::Params p{};
  p.pool = {a.code_pages, a.norm_pages, a.value_pages, a.num_pages, a.page_tokens,
            a.Hkv, a.words, a.norms_per_key, a.d, device_error_ptr()};
  if (!p.pool.err) return cudaErrorInvalidSymbol;
  p.mass = a.mass; p.lens = a.seq_lens; p.src_table = a.src_table; p.dst_table = a.dst_table;
  p.src_pages = a.src_max_pages; p.dst_pages = a.dst_max_pages; p.B = a.B; p.T = a.max_len;
  p.keep = a.keep; p.recent = a.recent; p.sink = a.sink;
  p.out_index = a.out_index; p.out_mass = a.out_mass; p.out_lens = a.out_lens;
  const int cluster = cluster_for((int64_t)a.B * a.Hkv, a.max_len, evict::THREADS);
  const int64_t share = (a.max_len + cluster - 1) / cluster;
  // 192 KB of sort keys at most: with the block's static shared memory that
  // stays inside the 227 KB a block may have
  p.cached = evict::place(share) * 4 <= 192 * 1024;
  const size_t smem = p.cached ? (size_t)evict::place(share) * 4 : 0;
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024)  // with the static part, beyond what a block gets without asking
    e = cudaFuncSetAttribute(evict::select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             192 * 1024);
  if (e != cudaSuccess) return e;
  e = launch_cluster(evict::select_kernel, (int64_t)a.B * a.Hkv * cluster, cluster,
                     evict::THREADS, smem, stream, p);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(evict_blocks(a.keep) * a.B * a.Hkv));
  cfg.blockDim = dim3(evict::COPY_THREADS);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool four = a.words % 4 == 0;
  return cudaLaunchKernelEx(
      &cfg,
      a.d == 128 ? (four ? evict::move_kernel<128, 4> : evict::move_kernel<128, 1>)
                 : (four ? evict::move_kernel<64, 4> : evict::move_kernel<64, 1>),
      p);
}

}  // namespace jlk
