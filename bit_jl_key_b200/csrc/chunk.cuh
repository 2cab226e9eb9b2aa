// chunk.cuh -- what the two chunk attention kernels share: the plan of the
// work, the walk through a block's share of it, and the joining of split rows.
//
// Rows.  The query heads of a KV head share its keys, so row i * G + g of a
// (sequence, KV head) is token i, head g.  `rows` consecutive rows make a row
// tile, BN keys a key tile; a (row tile, key tile) pair that the row tile's
// last token sees is a unit.  Units are counted in the order (sequence, KV
// head, row tile, key tile) and every block takes an equal run of them, so a
// long context with few rows is split and many rows are balanced, the causal
// triangle included.  A row tile that lies in one block is written out by it;
// of a split one each block leaves the softmax states (acc, max, sum), and the
// last block to do so joins them, in the order of the keys.
#pragma once

#include "jl_common.cuh"
#include "jl_internal.h"

#include <cudaTypedefs.h>

namespace jlk {
namespace chunk {

constexpr int BN = 128;            // keys of a tile
// log2 of the largest weight before a row's maximum is renewed: far below what
// a weight, a sum of them or a value times them can be, and seldom reached
constexpr float RENEW = 16.f;
constexpr float MIN_SCALE = 1.17549435e-38f;  // of a row: -inf times it stays -inf
constexpr int PREP_THREADS = 256;
constexpr int SM_COUNT = 148;      // bounds the workspace per shape
constexpr int MOST_RECORDS = 128;  // states of one split row tile
constexpr int MIN_UNITS = 2;       // of a block: less is not worth another state to join

struct Plan {
  int64_t quota;      // units (key tiles, at least one per row tile) per block
};
struct Start {        // where a block's run begins
  int64_t u, end;     // units [u, end); none where u >= end
  int b, h, mt, k0;   // the unit u: sequence, KV head, row tile, unit of it
  int n, L, row, units;  // the sequence's tokens, keys, first row; units of the row tile
};
struct Work {         // workspace
  Plan *plan;
  Start *begin;       // [blocks]
  int64_t *b_unit;    // [B + 1] first unit of each sequence
  int32_t *b_tile;    // [B] first entry of its row tiles in mt_pre
  int32_t *start, *count, *len;  // [B] first row, tokens, keys, made safe
  int32_t *mt_pre;    // per sequence: units before each row tile of a head, and their sum
  uint16_t *U;        // [Hkv][N G][K] binary16 queries, scaled row by row
  float *rs;          // [Hkv][N G] row scale: log2 units per unit of score
  float *part;        // [2 blocks] softmax states: a block's first and last row tile
  int32_t *arrived;   // [2 blocks] states left of the split row tile that begins in a block
  uint16_t *keys;     // [B][Hkv][tiles of max_len][BN][d] binary16 keys (many rows)
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
  int B, Hq, Hkv, G, P, max_pages, num_pages, blocks, rows;
  int key_tiles;      // of max_len
  int gran, gran_log; // keys of a tile copied at once, all in one page: 32, 64 or 128
  int64_t N, max_len;
  float scale;        // softmax_scale
  int *err;
};

// Units of row tile mt: key tiles that its last token sees, at least one.
__device__ __forceinline__ int tile_units(int mt, int n, int L, int G, int rows) {
  const int last = min(n - 1, (rows * mt + rows - 1) / G);
  const int seen = max(0, L - n + last + 1);
  return max(1, (seen + BN - 1) / BN);
}

__device__ __forceinline__ void make_plan(const Params &p) {
  __shared__ int64_t units[PREP_THREADS];  // of a head, then before the sequence
  __shared__ int tiles[PREP_THREADS];
  __shared__ int first[PREP_THREADS], tokens[PREP_THREADS], keys[PREP_THREADS];
  __shared__ int64_t u_done;
  __shared__ int t_done, rows_done, longest;  // longest: key tiles of a sequence
  if (threadIdx.x == 0) {
    u_done = 0;
    t_done = rows_done = longest = 0;
  }
  __syncthreads();
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
      nt = (int)(((int64_t)n * p.G + p.rows - 1) / p.rows);
      for (int mt = 0; mt < nt; ++mt) tot += tile_units(mt, n, L, p.G, p.rows);
      if (nt) atomicMax(&longest, (L + BN - 1) / BN);
    }
    units[threadIdx.x] = tot;
    tiles[threadIdx.x] = nt ? nt + 1 : 0;
    first[threadIdx.x] = (int)c0;
    tokens[threadIdx.x] = n;
    keys[threadIdx.x] = L;
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
      if (nt && !JL_IN_RANGE(p.err, tiles[threadIdx.x], nt + 1,
                             p.N * p.G / p.rows + 2 * (int64_t)p.B + 1))
        nt = 0;
      for (int mt = 0; mt < nt; ++mt) {
        pre[mt] = u;
        u += tile_units(mt, n, L, p.G, p.rows);
      }
      if (nt) pre[nt] = u;
    }
    __syncthreads();
  }
  const int64_t total = u_done;
  int64_t quota = (total + p.blocks - 1) / p.blocks;
  if (quota < MIN_UNITS) quota = MIN_UNITS;
  // a row tile is split over MOST_RECORDS blocks at most
  if (quota < longest / (MOST_RECORDS - 2) + 1) quota = longest / (MOST_RECORDS - 2) + 1;
  if (threadIdx.x == 0) {
    p.w.b_unit[p.B] = total;
    p.w.plan->quota = quota;
  }
  __threadfence_block();
  __syncthreads();
  // where each block begins; up to PREP_THREADS sequences are still at hand in
  // shared memory, and so is a row tile of the first few of a sequence
  const bool here = p.B <= PREP_THREADS;
  for (int i = threadIdx.x; i < p.blocks; i += PREP_THREADS) {
    p.w.arrived[2 * i] = p.w.arrived[2 * i + 1] = 0;
    Start s{};
    s.u = i * quota;
    s.end = s.u + quota < total ? s.u + quota : total;
    if (s.u < total) {
      auto first_unit = [&](int b) {
        return b == p.B ? total : here ? units[b] : p.w.b_unit[b];
      };
      int lo = 0, hi = p.B;  // the last b whose first unit is not above u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_unit(mid) <= s.u) lo = mid; else hi = mid;
      }
      s.b = lo;
      s.n = here ? tokens[lo] : p.w.count[lo];
      s.L = here ? keys[lo] : p.w.len[lo];
      s.row = here ? first[lo] : p.w.start[lo];
      const int64_t u0 = first_unit(lo), per_head = (first_unit(lo + 1) - u0) / p.Hkv;
      s.h = (int)((s.u - u0) / per_head);
      const int rem = (int)(s.u - u0 - s.h * per_head);
      const int nt = (int)(((int64_t)s.n * p.G + p.rows - 1) / p.rows);
      int a = 0, before = 0;
      if (nt <= 16) {
        s.units = tile_units(0, s.n, s.L, p.G, p.rows);
        while (before + s.units <= rem) {
          before += s.units;
          s.units = tile_units(++a, s.n, s.L, p.G, p.rows);
        }
      } else {
        const int32_t *pre = p.w.mt_pre + (here ? tiles[lo] : p.w.b_tile[lo]);
        int z = nt;
        while (z - a > 1) {
          const int mid = (a + z) >> 1;
          if (pre[mid] <= rem) a = mid; else z = mid;
        }
        before = pre[a];
        s.units = pre[a + 1] - before;
      }
      s.mt = a;
      s.k0 = rem - before;
    }
    p.w.begin[i] = s;
  }
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

// Whatever prep writes is read with __ldcg here: attend may start before prep
// ends and waits for it (griddep_wait), and a load declared read-only (__ldg)
// may be moved above that wait.

// A block's run of units, one row tile after another.
struct Seg {
  int b, h, mt, nt;   // sequence, KV head, row tile, row tiles of the sequence
  int k0, k1, units;  // its units [k0, k1) of `units`
  int n, L, start;    // the sequence's tokens, keys, first row
  int nk;             // key tiles to do: 0 where the row tile sees no key
  int64_t u, end;     // next unit, end of the run
};

__device__ __forceinline__ void seg_fill(Seg &s, const Params &p) {
  const int64_t left = s.end - s.u;
  s.k1 = (int)(left < s.units - s.k0 ? s.k0 + left : s.units);
  const int last = min(s.n - 1, (p.rows * s.mt + p.rows - 1) / p.G);
  s.nk = s.L - s.n + last + 1 > 0 ? s.k1 - s.k0 : 0;
}
__device__ __forceinline__ void seg_seq(Seg &s, const Params &p) {
  s.n = __ldcg(p.w.count + s.b);
  s.L = __ldcg(p.w.len + s.b);
  s.start = __ldcg(p.w.start + s.b);
  s.nt = (int)(((int64_t)s.n * p.G + p.rows - 1) / p.rows);
}
// First segment of the block; false when it has none.
__device__ __forceinline__ bool seg_first(Seg &s, const Params &p) {
  const int4 *q = reinterpret_cast<const int4 *>(p.w.begin + blockIdx.x);
  const int4 x = __ldcg(q), y = __ldcg(q + 1), z = __ldcg(q + 2);
  s.u = (int64_t)(((uint64_t)(uint32_t)x.y << 32) | (uint32_t)x.x);
  s.end = (int64_t)(((uint64_t)(uint32_t)x.w << 32) | (uint32_t)x.z);
  s.b = y.x; s.h = y.y; s.mt = y.z; s.k0 = y.w;
  s.n = z.x; s.L = z.y; s.start = z.z; s.units = z.w;
  s.nt = (int)(((int64_t)s.n * p.G + p.rows - 1) / p.rows);
  if (s.u >= s.end) return false;
  seg_fill(s, p);
  return true;
}
__device__ __forceinline__ bool seg_next(Seg &s, const Params &p) {
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
  const int32_t *pre = p.w.mt_pre + __ldcg(p.w.b_tile + s.b) + s.mt;
  s.units = __ldcg(pre + 1) - __ldcg(pre);
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

// ---------------------------------------------------------------------------
// split row tiles

// The blocks whose runs the segment's row tile touches, and where each of them
// leaves its states: record 2 c + 1 where block c has the row tile's first
// unit, 2 c otherwise (then the row tile is the first of its run).
struct Split {
  int64_t c0, c1, first, quota;
  __device__ __forceinline__ Split(const Seg &s, const Params &p) {
    quota = __ldcg(&p.w.plan->quota);
    first = s.u - s.k0;
    c0 = first / quota;
    c1 = (first + s.units - 1) / quota;
  }
  __device__ __forceinline__ int64_t record(int64_t c) const {
    return 2 * c + (c * quota <= first ? 1 : 0);
  }
};

// Called by `threads` threads that share the row tile (or half `a` of it),
// after each has written its part of the states: true, for all of them, in the
// last block to arrive. `flag` is a word of shared memory of theirs.
__device__ __forceinline__ bool last_to_arrive(const Split &t, const Params &p, int a, int bar,
                                               int threads, bool leader, volatile int *flag) {
  __threadfence();
  asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "r"(threads) : "memory");
  if (leader)
    *flag = atomicAdd(p.w.arrived + 2 * t.c0 + a, 1) == (int)(t.c1 - t.c0);
  asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "r"(threads) : "memory");
  const bool last = *flag != 0;
  if (last) __threadfence();
  return last;
}

// ---------------------------------------------------------------------------
// host

template <typename... Args>
inline cudaError_t launch_after(void (*kernel)(Args...), int64_t grid, int threads, size_t smem,
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


// The workspace: `rows` per row tile, K entries of a converted query, `part`
// floats of states per record, `keys` bytes of expanded keys.
inline size_t lay_out(Work *w, void *base, int64_t N, int B, int Hq, int Hkv, int rows, int K,
                      size_t part, size_t keys) {
  size_t off = 0;
  auto take = [&](size_t n) {
    uint8_t *x = static_cast<uint8_t *>(base) + off;
    off += (n + 255) & ~(size_t)255;
    return x;
  };
  Work t;
  t.plan = reinterpret_cast<Plan *>(take(sizeof(Plan)));
  t.begin = reinterpret_cast<Start *>(take((size_t)SM_COUNT * sizeof(Start)));
  t.b_unit = reinterpret_cast<int64_t *>(take((size_t)(B + 1) * 8));
  t.b_tile = reinterpret_cast<int32_t *>(take((size_t)B * 4));
  t.start = reinterpret_cast<int32_t *>(take((size_t)B * 4));
  t.count = reinterpret_cast<int32_t *>(take((size_t)B * 4));
  t.len = reinterpret_cast<int32_t *>(take((size_t)B * 4));
  t.mt_pre = reinterpret_cast<int32_t *>(
      take(((size_t)N * (Hq / Hkv) / rows + 2 * (size_t)B + 1) * 4));
  t.arrived = reinterpret_cast<int32_t *>(take((size_t)2 * SM_COUNT * 4));
  t.U = reinterpret_cast<uint16_t *>(take((size_t)N * Hq * K * 2));
  t.rs = reinterpret_cast<float *>(take((size_t)N * Hq * 4));
  t.part = reinterpret_cast<float *>(take((size_t)2 * SM_COUNT * part * 4));
  t.keys = reinterpret_cast<uint16_t *>(take(keys));
  if (w) *w = t;
  return off;
}

// A tile's values in shared memory: granule after granule, each as D / 64 boxes
// of gran rows x 128 bytes (64 dims, 128-byte swizzle), brought by one bulk
// tensor copy from the pool seen as [D / 64][rows][64].
inline bool make_value_map(CUtensorMap *map, const uint16_t *values, uint64_t rows, int d,
                           int gran) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  cuuint64_t dims[3] = {64, rows, (cuuint64_t)d / 64};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)gran, (cuuint32_t)d / 64};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(values), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Byte offset of key r of a tile in it (its first 64 dims); the others follow
// gran * 128 bytes apart.
__device__ __forceinline__ uint32_t value_offset(int r, const Params &p, int D) {
  const int g = r >> p.gran_log;
  return (uint32_t)((g << p.gran_log) * D * 2 + (r & (p.gran - 1)) * 128);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// The kernels for few and for many rows (chunk_few.cu, chunk_tc.cu): the
// workspace they need, and their launches.
size_t few_workspace(int64_t N, int B, int Hq, int Hkv, int m, int d, Work *w, void *base);
size_t many_workspace(int64_t N, int B, int Hq, int Hkv, int64_t max_len, int d, Work *w,
                      void *base);
cudaError_t launch_few(Params p, const ChunkArgs &a, cudaStream_t stream);
cudaError_t launch_many(Params p, const ChunkArgs &a, cudaStream_t stream);
constexpr int FEW_ROWS_LEAST = 32, FEW_ROWS_MOST = 64, MANY_ROWS = 256;  // of a row tile
int few_rows(int64_t N, int B, int G);  // which of the first two

}  // namespace chunk
}  // namespace jlk
