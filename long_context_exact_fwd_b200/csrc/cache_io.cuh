// Writing new keys and values into the cache's pages, and reading them back as bf16.
//
// Append: one block per (touched page, head, keys or values).  It holds the page's new rows in
// registers, takes their largest finite magnitude, and with it the page's exponent
//   e = max(e of the page if it holds older tokens, exponent of amax),
// restates the older codes if e grew, and writes RN_e4m3(x * 2^-e).  A scale never shrinks while
// its page holds tokens, so appending again over the same positions changes nothing.  What is not
// finite is stored as NaN and does not count into the scale.  Bound: memory, 2 bytes in and 1 out
// per element (one pass: amax and rounding from the same registers).
#pragma once
#include "cache.cuh"

namespace ra {
namespace cache {

constexpr int IO_THREADS = 256;
constexpr int UNIT = 16;      // elements of a thread's unit: 32 bytes of bf16, 16 of codes

struct AppendParams {
  Pool c;                      // one layer
  const __nv_bfloat16 *k, *v;  // [B][heads][T][Dh], strides in elements
  long long kb, kh, kt, vb, vh, vt;
  const int *slots, *n_new;    // n_new null: T
  int T;
};

struct Elems {
  uint4 a, b;                  // 16 bf16
};

__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x <= 3.4028234663852886e38f ? x : 0.f;   // not finite: 0
}
__device__ __forceinline__ uint32_t quantise4(uint32_t w0, uint32_t w1, float inv) {
  constexpr float TOP = 240.f * 1.329227995784916e36f;   // 240 * 2^120: all a code and scale can hold
  float x[4];
  unpack2(w0, x[0], x[1]);
  unpack2(w1, x[2], x[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = fminf(fmaxf(x[i], -TOP), TOP) * inv;
    x[i] = fabsf(x[i]) <= 3.4028234663852886e38f ? y : __uint_as_float(0x7fffffffu);
  }
  return floats_to_codes(x[0], x[1]) | (floats_to_codes(x[2], x[3]) << 16);
}
__device__ __forceinline__ uint32_t restate4(uint32_t codes, float f) {
  const float2 a = half2_to_float2(codes_to_half2(static_cast<uint16_t>(codes)));
  const float2 b = half2_to_float2(codes_to_half2(static_cast<uint16_t>(codes >> 16)));
  return floats_to_codes(a.x * f, a.y * f) | (floats_to_codes(b.x * f, b.y * f) << 16);
}

// NU: units per thread, ceil(page * Dh / UNIT / IO_THREADS).
template <int NU>
__global__ void __launch_bounds__(IO_THREADS) append_kernel(const AppendParams p) {
  const Pool& c = p.c;
  const int b = blockIdx.z >> 1, kv = blockIdx.z & 1, h = blockIdx.y;
  const int slot = p.slots[b];
  if (slot == -1) return;                         // a row of padding
  const bool reports = blockIdx.x == 0 && threadIdx.x == 0;
  if (slot < 0 || slot >= c.slots) {
    if (reports) record_status(RA_ERR_PAGES);
    return;
  }
  const int n = p.n_new ? p.n_new[b] : p.T;
  const int len = c.lens[slot];
  const int p0 = len - n;                         // first new position
  if (n < 0 || n > p.T || p0 < 0 || len > c.max_pages * static_cast<long long>(c.page)) {
    if (reports) record_status(RA_ERR_PAGES);
    return;
  }
  const int j = p0 / c.page + blockIdx.x;         // the page's place in the table
  const long long at0 = static_cast<long long>(j) * c.page;
  if (n == 0 || at0 >= len) return;
  const int pid = c.table[static_cast<long long>(slot) * c.max_pages + j];
  bool bad = pid < 0 || pid >= c.pages;
  if (!bad) bad = c.refs[pid] != 1;               // a page that others hold too is not written
  if (bad) {
    if (threadIdx.x == 0) record_status(RA_ERR_PAGES);
    return;
  }
  const __nv_bfloat16* src = (kv ? p.v : p.k) + b * (kv ? p.vb : p.kb) + h * (kv ? p.vh : p.kh);
  const long long st = kv ? p.vt : p.kt;
  const long long page_at = (static_cast<long long>(pid) * c.heads + h) * c.page * c.Dh;
  uint8_t* codes = (kv ? c.v : c.k) + page_at;
  float* scale = (kv ? c.v_scale : c.k_scale) + static_cast<long long>(pid) * c.heads + h;
  const int skip = max(0, static_cast<int>(p0 - at0));                       // older tokens in the page
  const int end = static_cast<int>(min(static_cast<long long>(c.page), len - at0));
  const int per_row = c.Dh / UNIT;

  Elems x[NU];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = threadIdx.x + i * IO_THREADS;
    const int t = u / per_row;
    if (t >= skip && t < end) {
      const uint4* q = reinterpret_cast<const uint4*>(src + (at0 + t - p0) * st + (u - t * per_row) * UNIT);
      x[i].a = q[0];
      x[i].b = q[1];
    } else {
      x[i].a = x[i].b = make_uint4(0, 0, 0, 0);
    }
  }
  const float old_scale = skip ? *scale : 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t w[8] = {x[i].a.x, x[i].a.y, x[i].a.z, x[i].a.w, x[i].b.x, x[i].b.y, x[i].b.z, x[i].b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float lo, hi;
      unpack2(w[k], lo, hi);
      amax = fmaxf(amax, fmaxf(finite_abs(lo), finite_abs(hi)));
    }
  }
  // magnitudes order like their bits
  __shared__ unsigned s_max[IO_THREADS / 32];
  const unsigned wmax = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = wmax;
  if (named_before(p.slots, b, slot)) {           // barrier: s_max and every read of the old scale
    if (reports) record_status(RA_ERR_PAGES);
    return;
  }
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < IO_THREADS / 32; ++i) m = max(m, s_max[i]);
  int e = scale_exponent(__uint_as_float(m));
  int e_old = e;
  if (skip) {
    e_old = min(max(exponent_of(old_scale), E_MIN), E_MAX);
    e = max(e, e_old);
  }
  const float inv = two_to(-e);
  const float shrink = two_to(max(e_old - e, -126));
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = threadIdx.x + i * IO_THREADS;
    const int t = u / per_row;
    uint4* dst = reinterpret_cast<uint4*>(codes) + u;
    if (t >= skip && t < end) {
      *dst = make_uint4(quantise4(x[i].a.x, x[i].a.y, inv), quantise4(x[i].a.z, x[i].a.w, inv),
                        quantise4(x[i].b.x, x[i].b.y, inv), quantise4(x[i].b.z, x[i].b.w, inv));
    } else if (t < skip && e > e_old) {
      const uint4 o = *dst;
      *dst = make_uint4(restate4(o.x, shrink), restate4(o.y, shrink), restate4(o.z, shrink), restate4(o.w, shrink));
    }
  }
  if (threadIdx.x == 0) *scale = two_to(e);
}

struct ReadParams {
  Pool c;                      // one layer
  const int *slots, *start;    // start null: 0
  __nv_bfloat16 *k, *v;        // [B][heads][length][Dh]
  int length;
};

// Positions start .. start + length - 1 of each sequence; zero behind its end (and before 0).
__global__ void __launch_bounds__(IO_THREADS) read_kernel(const ReadParams p) {
  const Pool& c = p.c;
  const int b = blockIdx.z >> 1, kv = blockIdx.z & 1, h = blockIdx.y;
  const int slot = p.slots[b];
  if (slot == -1) return;
  if (slot < 0 || slot >= c.slots) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_status(RA_ERR_PAGES);
    return;
  }
  const int per_row = c.Dh / UNIT;
  const long long u = static_cast<long long>(blockIdx.x) * IO_THREADS + threadIdx.x;
  const long long t = u / per_row;
  if (t >= p.length) return;
  const long long pos = (p.start ? p.start[b] : 0) + t;
  const int col = static_cast<int>(u - t * per_row) * UNIT;
  uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (pos >= 0 && pos < c.lens[slot] && pos < c.max_pages * static_cast<long long>(c.page)) {
    const int pid = c.table[static_cast<long long>(slot) * c.max_pages + pos / c.page];
    if (pid < 0 || pid >= c.pages) {
      record_status(RA_ERR_PAGES);
    } else {
      const long long ph = static_cast<long long>(pid) * c.heads + h;
      const uint4 w = *reinterpret_cast<const uint4*>((kv ? c.v : c.k) + (ph * c.page + pos % c.page) * c.Dh + col);
      const float s = (kv ? c.v_scale : c.k_scale)[ph];
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = half2_to_float2(codes_to_half2(static_cast<uint16_t>(in[i])));
        const float2 hi = half2_to_float2(codes_to_half2(static_cast<uint16_t>(in[i] >> 16)));
        out[2 * i] = pack_bf16x2(lo.x * s, lo.y * s);
        out[2 * i + 1] = pack_bf16x2(hi.x * s, hi.y * s);
      }
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((kv ? p.v : p.k) +
                                        ((static_cast<long long>(b) * c.heads + h) * p.length + t) * c.Dh + col);
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

}  // namespace cache
}  // namespace ra
