// rotary.cu -- rotary positions on the queries and keys of a step, ahead of
// the quantizer and of decode.
//
// Pair j of a head (entries j and j + r/2 in the half layout, 2j and 2j + 1 in
// the interleaved one, j < r/2) turns by the angle a = pos * f_j:
//     (x, y) -> scale * (x cos a - y sin a, x sin a + y cos a),
// the inverse (and, the rotation being orthogonal, the gradient) by -a; entries
// from r on are copied.
//
// The angle is formed and reduced to [-pi, pi] in 64 bits: at position 2^20 an
// fp32 product is already off by up to 2^-5 radians.  The reduced angle's fp32
// rounding is put back to first order (sin(t + e) = sin t + e cos t), so cos
// and sin carry about 1e-7 whatever the position.
//
// Bound by memory: every entry is read and written once and a pair costs four
// multiply-adds, so what matters is that a token's angles are computed once
// for all its heads.  A block takes `tok` tokens and a range of heads, puts
// their (cos, sin) into shared memory, then streams the heads with 16-byte
// loads and stores.  Measured: 16384 tokens of 40 heads (d = 128, 64 of them
// turned, bf16) are 336 MB in 63.9 us, 5.25 TB/s; a decode step of 8 tokens is one
// launch, 2.2 us in a graph.
#include "jl_common.cuh"
#include "jl_internal.h"

namespace jlk {
namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_TOK = 8;

struct Side {  // one of queries and keys: strides in elements
  const void *x;
  void *y;
  int64_t x_tok, x_head, y_tok, y_head;
};

struct Params {
  Side q, k;
  int Hq, H;  // query heads; query and key heads together
  int64_t n;
  int d, rot, tok, heads_per_block;
  uint64_t units_inv, heads_inv;  // of a head's units and of a block's heads (see over())
  const int32_t *pos;
  const float *inv_freq;
  float scale, sign;
  int *err;
};

// a / b from ceil(2^40 / b), without a division (which per 16 bytes moved is what
// bound this kernel): exact while a * b < 2^40, and a block has at most
// MAX_TOK * MAX_HEADS * 1024 units of at most 1024 per head.
constexpr int MAX_HEADS = 1024;
static_assert((uint64_t)MAX_TOK * MAX_HEADS * 1024 * 1024 < (1ull << 40), "exact quotients");
__host__ __device__ __forceinline__ uint64_t inverse_of(uint32_t b) {
  return ((1ull << 40) + b - 1) / b;
}
__device__ __forceinline__ int over(int a, uint64_t inv) {
  return (int)(((uint64_t)(uint32_t)a * inv) >> 40);
}

// Elements a side's tensor spans (index checks of the debug build).
__device__ __forceinline__ int64_t span(int64_t n, int H, int d, int64_t tok, int64_t head) {
  return (n - 1) * tok + (H - 1) * head + d;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_bits_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// VEC consecutive entries (16 bytes where VEC * sizeof(T) is 16)
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load(const T *p) {
  Pack<T, VEC> r;
  if constexpr (sizeof(T) * VEC == 16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    memcpy(&r, &u, 16);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) r.v[i] = p[i];
  }
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T *p, const Pack<T, VEC> &r) {
  if constexpr (sizeof(T) * VEC == 16) {
    uint4 u;
    memcpy(&u, &r, 16);
    *reinterpret_cast<uint4 *>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = r.v[i];
  }
}

// A unit is what one thread turns at a time.  Half layout: VEC entries of the
// first half and their partners; interleaved: VEC consecutive entries (VEC / 2
// pairs).  Units past the rotated part copy VEC entries.
template <typename T, bool INTER, int VEC>
__global__ void __launch_bounds__(THREADS) rotary_kernel(const Params p) {
  extern __shared__ float2 cs[];  // [tok][rot / 2]
  const int half = p.rot >> 1;
  const int64_t t0 = (int64_t)blockIdx.x * p.tok;
  const int toks = (int)(p.n - t0 < p.tok ? p.n - t0 : p.tok);
  for (int i = threadIdx.x; i < toks * half; i += THREADS) {
    const int tk = i / half, j = i - tk * half;
    if (!JL_IN_RANGE(p.err, t0 + tk, 1, p.n) || !JL_IN_RANGE(p.err, j, 1, half)) continue;
    const double a = (double)p.pos[t0 + tk] * (double)p.inv_freq[j];
    // a - 2 pi k with 2 pi in two parts
    const double k = rint(a * 0.15915494309189533577);
    double r = fma(-k, 6.28318530717958623200, a);
    r = fma(-k, 2.44929359829470635e-16, r);
    const float rf = (float)r, e = (float)(r - (double)rf);
    float s, c;
    sincosf(rf, &s, &c);
    const float s1 = fmaf(e, c, s), c1 = fmaf(-e, s, c);
    cs[i] = make_float2(c1 * p.scale, s1 * p.sign * p.scale);
  }
  __syncthreads();

  const int ru = INTER ? p.rot / VEC : half / VEC;   // turning units of a head
  const int units = ru + (p.d - p.rot) / VEC;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int nh = p.H - h0 < p.heads_per_block ? p.H - h0 : p.heads_per_block;
  const int total = toks * nh * units;
  // (the last blocks of a row have fewer heads than the others)
  const uint64_t nh_inv = nh == p.heads_per_block ? p.heads_inv : inverse_of(nh);
  constexpr int AT_ONCE = 4;  // units of a thread whose loads are in flight together
  for (int i0 = threadIdx.x; i0 < total; i0 += THREADS * AT_ONCE) {
    Pack<T, VEC> v[AT_ONCE], w[AT_ONCE];
    T *y[AT_ONCE];
    int tk[AT_ONCE], u[AT_ONCE];
#pragma unroll
    for (int q = 0; q < AT_ONCE; ++q) {
      const int i = i0 + q * THREADS;
      if (i >= total) {
        u[q] = -1;
        continue;
      }
      const int row = over(i, p.units_inv);
      u[q] = i - row * units;
      tk[q] = over(row, nh_inv);
      const int h = h0 + row - tk[q] * nh;
      const bool is_q = h < p.Hq;
      const Side &s = is_q ? p.q : p.k;
      const int hh = is_q ? h : h - p.Hq;
      const T *x = static_cast<const T *>(s.x) + (t0 + tk[q]) * s.x_tok + hh * s.x_head;
      y[q] = static_cast<T *>(s.y) + (t0 + tk[q]) * s.y_tok + hh * s.y_head;
      const int o = u[q] < ru ? u[q] * VEC : p.rot + (u[q] - ru) * VEC;
      const int last = (!INTER && u[q] < ru ? half : 0) + o + VEC;  // of the row's entries
      const int Hs = is_q ? p.Hq : p.H - p.Hq;
      if (!JL_IN_RANGE(p.err, (t0 + tk[q]) * s.x_tok + hh * s.x_head, last,
                       span(p.n, Hs, p.d, s.x_tok, s.x_head)) ||
          !JL_IN_RANGE(p.err, (t0 + tk[q]) * s.y_tok + hh * s.y_head, last,
                       span(p.n, Hs, p.d, s.y_tok, s.y_head))) {
        u[q] = -1;
        continue;
      }
      y[q] += o;
      v[q] = load<T, VEC>(x + o);
      if (!INTER && u[q] < ru) w[q] = load<T, VEC>(x + half + o);
    }
#pragma unroll
    for (int q = 0; q < AT_ONCE; ++q) {
      if (u[q] < 0) continue;
      if (u[q] < ru) {
        const float2 *r = cs + tk[q] * half;
        if constexpr (INTER) {
          r += u[q] * (VEC / 2);
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float a = to_f32(v[q].v[e]), b = to_f32(v[q].v[e + 1]);
            v[q].v[e] = from_f32<T>(fmaf(a, r[e / 2].x, -b * r[e / 2].y));
            v[q].v[e + 1] = from_f32<T>(fmaf(a, r[e / 2].y, b * r[e / 2].x));
          }
        } else {
          r += u[q] * VEC;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float a = to_f32(v[q].v[e]), b = to_f32(w[q].v[e]);
            v[q].v[e] = from_f32<T>(fmaf(a, r[e].x, -b * r[e].y));
            w[q].v[e] = from_f32<T>(fmaf(a, r[e].y, b * r[e].x));
          }
          store<T, VEC>(y[q] + half, w[q]);
        }
      }
      store<T, VEC>(y[q], v[q]);
    }
  }
}

template <typename T, bool INTER, int VEC>
cudaError_t launch_t(Params p, cudaStream_t stream) {
  // Tokens per block: enough units to occupy the threads, shared angles for
  // all heads; few tokens spread their heads over more blocks instead.
  const int sms = device_sm_count();
  int tok = 1;
  while (tok < MAX_TOK && p.n / (2 * tok) >= 4 * sms) tok *= 2;
  p.tok = tok;
  const int64_t gx = (p.n + tok - 1) / tok;
  int split = 1;
  while (split < p.H && gx * split < 2 * sms && split < 64) ++split;
  p.heads_per_block = (p.H + split - 1) / split;
  if (p.heads_per_block > MAX_HEADS) p.heads_per_block = MAX_HEADS;
  const int ru = INTER ? p.rot / VEC : p.rot / 2 / VEC;
  p.units_inv = inverse_of(ru + (p.d - p.rot) / VEC);
  p.heads_inv = inverse_of(p.heads_per_block);
  const int gy = (p.H + p.heads_per_block - 1) / p.heads_per_block;
  const size_t smem = (size_t)tok * (p.rot / 2) * sizeof(float2);
  rotary_kernel<T, INTER, VEC><<<dim3((unsigned)gx, gy), THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_v(const Params &p, bool inter, cudaStream_t stream) {
  // 16-byte units where every row starts on 16 bytes and the rotated part is
  // whole units; otherwise entry by entry (pairs when interleaved)
  constexpr int V = 16 / (int)sizeof(T);
  auto ok = [](const Side &s) {
    if (!s.x) return true;
    const uint64_t a = (uint64_t)reinterpret_cast<uintptr_t>(s.x) |
                       (uint64_t)reinterpret_cast<uintptr_t>(s.y) |
                       (uint64_t)(s.x_tok | s.x_head | s.y_tok | s.y_head) * sizeof(T);
    return (a & 15) == 0;
  };
  const int part = inter ? p.rot : p.rot / 2;
  const bool vec = part % V == 0 && p.rot % V == 0 && p.d % V == 0 && ok(p.q) && ok(p.k);
  if (inter) return vec ? launch_t<T, true, V>(p, stream) : launch_t<T, true, 2>(p, stream);
  return vec ? launch_t<T, false, V>(p, stream) : launch_t<T, false, 1>(p, stream);
}

}  // namespace rope

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t stream) {
  rope::Params p{};
  p.q = {a.q, a.out_q, a.q_tok, a.q_head, a.out_q_tok, a.out_q_head};
  p.k = {a.k, a.out_k, a.k_tok, a.k_head, a.out_k_tok, a.out_k_head};
  p.Hq = a.Hq;
  p.H = a.Hq + (a.k ? a.Hkv : 0);
  p.n = a.n;
  p.d = a.d;
  p.rot = a.rot;
  p.pos = a.positions;
  p.inv_freq = a.inv_freq;
  p.scale = a.scale;
  p.sign = a.inverse ? -1.f : 1.f;
  p.err = device_error_ptr();
  if (!p.err) return cudaErrorInvalidSymbol;
  return a.f32 ? rope::launch_v<float>(p, a.interleaved, stream)
               : rope::launch_v<uint16_t>(p, a.interleaved, stream);
}

}  // namespace jlk
