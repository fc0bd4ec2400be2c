// Rotary positions: every pair (x1, x2) of the first `rot` columns of a head is turned by the
// angle a = position * theta_i and scaled by the plan's amplitude A:
//   y1 = A (x1 cos a - x2 sin a),   y2 = A (x1 sin a + x2 cos a);
// columns from `rot` on pass through.  The gradient is the inverse turn (sin -> -sin) with the
// same A.  Pairs are (2i, 2i + 1), or (i, i + rot / 2).
//
// Angles.  The plan holds theta_i / 2 pi as a 64-bit fixed-point fraction of a turn, so
// position * step mod 2^64 is the phase with whole turns dropped, exact in integer arithmetic:
// with a step to the nearest unit the error left is position * 2^-65 turns, at any position.  The phase is brought to the nearest
// quarter turn before it becomes a float (|r| <= 1/8 turn keeps 24 good bits).  No table is kept or
// read.
//
// Bound: memory (each element read and written once).  A thread owns one group of pairs of one
// token and walks over heads, so one sine and cosine serve `heads_per_thread` heads of Q and K.
// Measured on B200: 16384 tokens, 16 + 16 heads of 128, bf16: 49.1 us, 5.5 TB/s (84 % of a copy);
// 8198 tokens, 8 + 2 heads, 96 of 128 columns, interleaved float32: 13.2 us, 97 %.
#pragma once
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

namespace ra {
namespace rope {

constexpr int THREADS = 256;
// Heads that rope_rows_kernel loads before it stores the first, and by which rope_kernel's loop is unrolled (its
// stores may be to the next heads' inputs, for all that the compiler knows, so its loads stay behind them).
constexpr int HEADS_AT_ONCE = 4;

struct Tensor {               // one of Q, K: strides in elements, last dimension contiguous
  const void* x;
  void* y;
  long long xb, xh, xs, yb, yh, ys;
  int heads;
};

struct Params {
  Tensor t[2];                // heads of t[0], then of t[1] (heads 0: absent)
  const unsigned long long* steps;   // [rot / 2], theta / 2 pi in units of 2^-64 turn
  const long long* pos;       // or null: position = offset + s
  long long pos_b, pos_s, offset;
  long long tokens;           // B * S
  int wide_ids;               // tokens * units passes 32 bits
  int S, Dh, rot;
  int units;                  // groups of columns per token
  int rot_units;              // of them, groups that are rotated
  int heads_per_thread;
  float amplitude;
  int inverse;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// VECTOR: N elements move as one aligned access; otherwise one by one.
template <typename T, int N, bool VECTOR>
__device__ __forceinline__ void load(const T* p, T (&v)[N]) {
  if (VECTOR) {
    const Pack<T, N> a = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = a.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = p[i];
  }
}
template <typename T, int N, bool VECTOR>
__device__ __forceinline__ void store(T* p, const T (&v)[N]) {
  if (VECTOR) {
    Pack<T, N> a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = v[i];
    *reinterpret_cast<Pack<T, N>*>(p) = a;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = v[i];
  }
}

// Elements as floats and back, bf16 in pairs (one conversion instruction rounds two).
template <int N>
__device__ __forceinline__ void widen(const float (&a)[N], float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = a[i];
}
template <int N>
__device__ __forceinline__ void widen(const __nv_bfloat16 (&a)[N], float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __bfloat162float(a[i]);
}
template <int N>
__device__ __forceinline__ void narrow(const float (&f)[N], float (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = f[i];
}
template <int N>
__device__ __forceinline__ void narrow(const float (&f)[N], __nv_bfloat16 (&a)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[i], f[i + 1]);
      a[i] = v.x;
      a[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] = __float2bfloat16_rn(f[i]);
  }
}

// cos and sin of 2 pi * phase * 2^-64.  The phase is split into the nearest quarter turn and a rest
// r, |r| <= 1/8 turn; with t = 2 pi r the Taylor series cut at t^9 and t^10 are within 2e-9 and 2e-10
// for |t| <= pi / 4, below float's half step (sincospif, which reduces any argument, made the 16K-token
// prompt 10 % slower).
__device__ __forceinline__ void turn(unsigned long long phase, float& c, float& s) {
  const unsigned quarter = static_cast<unsigned>((phase + (1ull << 61)) >> 62) & 3u;
  const int r = static_cast<int>((phase - (static_cast<unsigned long long>(quarter) << 62)) >> 32);
  const float t = static_cast<float>(r) * 1.4629180792671596e-9f;   // 2 pi * 2^-32
  const float u = t * t;
  float sr = fmaf(u, 2.7557319223985893e-6f, -1.9841269841269841e-4f);   // 1/9!, -1/7!
  sr = fmaf(sr, u, 8.3333333333333333e-3f);
  sr = fmaf(sr, u, -1.6666666666666667e-1f);
  sr = fmaf(sr * u, t, t);
  float cr = fmaf(u, -2.7557319223985888e-7f, 2.4801587301587302e-5f);   // -1/10!, 1/8!
  cr = fmaf(cr, u, -1.3888888888888889e-3f);
  cr = fmaf(cr, u, 4.1666666666666667e-2f);
  cr = fmaf(cr, u, -0.5f);
  cr = fmaf(cr, u, 1.f);
  const float a = (quarter & 1u) ? sr : cr, b = (quarter & 1u) ? cr : sr;
  c = (quarter == 1u || quarter == 2u) ? -a : a;
  s = (quarter >= 2u) ? -b : b;
}

// A unit is N columns (interleaved: N / 2 pairs) or N columns and their N partners (half).
template <typename T, int N, bool INTERLEAVED, bool VECTOR>
__global__ void __launch_bounds__(THREADS) rope_kernel(const Params p) {
  const long long id = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
  const long long token = id / p.units;
  if (token >= p.tokens) return;
  const int unit = static_cast<int>(id - token * p.units);
  const long long b = token / p.S, s = token - b * p.S;
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int all = p.t[0].heads + p.t[1].heads;
  const int h1 = min(h0 + p.heads_per_thread, all);
  const bool rotated = unit < p.rot_units;
  constexpr int PAIRS = INTERLEAVED ? N / 2 : N;
  float c[PAIRS], sn[PAIRS];
  int col, col2 = 0;
  if (rotated) {
    const long long pos = p.pos ? p.pos[b * p.pos_b + s * p.pos_s] : p.offset + s;
    const int i0 = unit * PAIRS;
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      turn(static_cast<unsigned long long>(pos) * p.steps[i0 + i], c[i], sn[i]);
      c[i] *= p.amplitude;
      sn[i] *= p.inverse ? -p.amplitude : p.amplitude;
    }
    col = INTERLEAVED ? unit * N : i0;
    col2 = i0 + p.rot / 2;
  } else {
    col = p.rot + (unit - p.rot_units) * N;
  }
#pragma unroll HEADS_AT_ONCE
  for (int h = h0; h < h1; ++h) {
    const bool second = h >= p.t[0].heads;
    const Tensor& t = p.t[second ? 1 : 0];
    const int hh = second ? h - p.t[0].heads : h;
    const T* x = static_cast<const T*>(t.x) + b * t.xb + hh * t.xh + s * t.xs;
    T* y = static_cast<T*>(t.y) + b * t.yb + hh * t.yh + s * t.ys;
    T a[N];
    load<T, N, VECTOR>(x + col, a);
    if (!rotated) {
      if (y != x) store<T, N, VECTOR>(y + col, a);
      continue;
    }
    float f[N];
    widen<N>(a, f);
    if (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float x1 = f[2 * i], x2 = f[2 * i + 1];
        f[2 * i] = fmaf(x1, c[i], -x2 * sn[i]);
        f[2 * i + 1] = fmaf(x1, sn[i], x2 * c[i]);
      }
    } else {
      T a2[N];
      float f2[N];
      load<T, N, VECTOR>(x + col2, a2);
      widen<N>(a2, f2);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x1 = f[i], x2 = f2[i];
        f[i] = fmaf(x1, c[i], -x2 * sn[i]);
        f2[i] = fmaf(x1, sn[i], x2 * c[i]);
      }
      narrow<N>(f2, a2);
      store<T, N, VECTOR>(y + col2, a2);
    }
    narrow<N>(f, a);
    store<T, N, VECTOR>(y + col, a);
  }
}

// A thread's place: its token, and its unit of the row.
struct Place {
  long long token, b, s;
  int unit;
};
__device__ __forceinline__ Place place(const Params& p) {
  Place r;
  const long long id = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
  if (p.wide_ids) {
    r.token = id / p.units;
    r.b = r.token / p.S;
  } else {
    r.token = static_cast<unsigned>(id) / static_cast<unsigned>(p.units);
    r.b = static_cast<unsigned>(r.token) / static_cast<unsigned>(p.S);
  }
  r.unit = static_cast<int>(id - r.token * p.units);
  r.s = r.token - r.b * p.S;
  return r;
}
// Calls body(x, y, x's and y's distance from head to head, heads) for the block's heads of Q, then of K; x, y at
// column `col` of the first.
template <typename T, typename F>
__device__ __forceinline__ void each_tensor(const Params& p, const Place& at, int col, F body) {
  const int h0 = blockIdx.y * p.heads_per_thread, h1 = h0 + p.heads_per_thread;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const Tensor& t = p.t[i];
    const int before = i ? p.t[0].heads : 0;
    const int a = max(h0 - before, 0), n = min(h1 - before, t.heads) - a;
    if (n > 0)
      body(static_cast<const T*>(t.x) + at.b * t.xb + at.s * t.xs + a * t.xh + col,
           static_cast<T*>(t.y) + at.b * t.yb + at.s * t.ys + a * t.yh + col, t.xh, t.yh, n);
  }
}

// The same by whole rows, where a row starts at a vector: for pairs at any distance, and for interleaved ones.  A
// thread has one vector of a row; a half layout's partners, and its angles, come from the row's other threads
// through shared memory (they are in one warp; outputs may be the inputs, so a row is read before it is written).
// Measured, columns of a projection: half, float32, 38 of 128, 19516 tokens, 16 + 8 heads 74 us, 99 % of a copy
// (rope_kernel, element by element, 164); bf16, 30 of 64, 11710 tokens, 64 + 16 heads 48 us, 76 % (147).  Bound
// there by instructions: partners read as shifted words, with a branch for each half, took 72 us.
template <typename T, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_rows_kernel(const Params p) {
  __shared__ Pack<T, N> rows[INTERLEAVED ? 1 : THREADS / 32][INTERLEAVED ? 1 : HEADS_AT_ONCE][32];
  const Place at = place(p);
  if (at.token >= p.tokens) return;
  const int col = at.unit * N, half = p.rot / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool rotated = col < p.rot;
  float c[N], sn[N];                         // y = x c + partner sn
  int partner[N];                            // half: its place in the warp's rows
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int j = col + i;
    partner[i] = lane * N + i + (j < half ? half : j < p.rot ? -half : 0);
  }
  const long long pos = p.pos ? p.pos[at.b * p.pos_b + at.s * p.pos_s] : p.offset + at.s;
  auto angle = [&](int i, float& co, float& si) {
    turn(static_cast<unsigned long long>(pos) * p.steps[i], co, si);
    co *= p.amplitude;
    si *= p.inverse ? -p.amplitude : p.amplitude;
  };
  if constexpr (INTERLEAVED) {
    if (rotated) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        angle(min(col + i, p.rot - 1) / 2, c[i], sn[i + 1]);
        c[i + 1] = c[i];
        sn[i] = -sn[i + 1];
      }
    }
  } else {                                   // a row's threads share its angles out
    __shared__ float2 angles[THREADS / 32][16 * N];
    float2* mine = angles[warp] + (lane - at.unit) * (N / 2);
    for (int i = at.unit; i < half; i += p.units) angle(i, mine[i].x, mine[i].y);
    __syncwarp();
    if (rotated) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = min(col + i, p.rot - 1);
        const float2 cs = mine[j < half ? j : j - half];
        c[i] = cs.x;
        sn[i] = j < half ? -cs.y : cs.y;
      }
    }
  }
  each_tensor<T>(p, at, col, [&](const T* x, T* y, long long xh, long long yh, int n) {
    for (int h = 0; h < n; h += HEADS_AT_ONCE, x += HEADS_AT_ONCE * xh, y += HEADS_AT_ONCE * yh) {
      Pack<T, N> a[HEADS_AT_ONCE];
#pragma unroll
      for (int k = 0; k < HEADS_AT_ONCE; ++k)
        if (h + k < n) a[k] = *reinterpret_cast<const Pack<T, N>*>(x + k * xh);
      if constexpr (!INTERLEAVED) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < HEADS_AT_ONCE; ++k)
          if (h + k < n) rows[warp][k][lane] = a[k];
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < HEADS_AT_ONCE; ++k) {
        if (h + k >= n) break;
        if (rotated) {
          float f[N], z[N];
          widen<N>(a[k].v, f);
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = f[i ^ 1];
          } else {
            T other[N];
#pragma unroll
            for (int i = 0; i < N; ++i) other[i] = reinterpret_cast<const T*>(rows[warp][k])[partner[i]];
            widen<N>(other, z);
          }
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = fmaf(f[i], c[i], z[i] * sn[i]);
          Pack<T, N> r;
          narrow<N>(f, r.v);
          // rot is even, and so is col: pairs of columns are rotated together
          using Two = std::conditional_t<sizeof(T) == 2, uint32_t, uint2>;
#pragma unroll
          for (int i = 0; i < N; i += 2)
            if (col + i < p.rot) reinterpret_cast<Two*>(a[k].v)[i / 2] = reinterpret_cast<const Two*>(r.v)[i / 2];
        }
        if (rotated || x != y) *reinterpret_cast<Pack<T, N>*>(y + k * yh) = a[k];
      }
    }
  });
}

}  // namespace rope
}  // namespace ra
