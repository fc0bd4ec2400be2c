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
// Elements of a thread's unit: 16 bytes of bf16, 8 of codes, so that a warp's accesses are whole lines on
// both sides (32 and 16 bytes a thread left half of every sector out: reading back the 8K prompt took 41 us
// against 33).
constexpr int UNIT = 8;

struct AppendParams {
  Pool c;                      // one layer
  const __nv_bfloat16 *k, *v;  // [B][heads][T][Dh], strides in elements
  long long kb, kh, kt, vb, vh, vt;
  const int *slots, *n_new;    // n_new null: T
  int T;
};

__device__ __forceinline__ void unpack2(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
constexpr uint32_t BF16_INF = 0x7f80u;
// Magnitudes of two bf16, as the numbers that their bits are (they order alike); what is not finite
// counts as 0.
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  w &= 0x7fff7fffu;
  return __vcmpltu2(w, BF16_INF * 0x10001u) & w;
}
// EXACT_RANGE: elements that are not finite, or past 240 * 2^120 (all that a code and scale hold).
template <bool EXACT_RANGE>
__device__ __forceinline__ uint32_t quantise4(uint32_t w0, uint32_t w1, float inv) {
  float x[4];
  unpack2(w0, x[0], x[1]);
  unpack2(w1, x[2], x[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (EXACT_RANGE) {
      constexpr float TOP = 240.f * 1.329227995784916e36f;
      const float y = fminf(fmaxf(x[i], -TOP), TOP) * inv;
      x[i] = fabsf(x[i]) <= 3.4028234663852886e38f ? y : __uint_as_float(0x7fffffffu);
    } else {
      x[i] *= inv;
    }
  }
  return floats_to_codes(x[0], x[1]) | (floats_to_codes(x[2], x[3]) << 16);
}
template <bool EXACT_RANGE>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  return make_uint2(quantise4<EXACT_RANGE>(x.x, x.y, inv), quantise4<EXACT_RANGE>(x.z, x.w, inv));
}
__device__ __forceinline__ uint32_t restate4(uint32_t codes, float f) {
  const float2 a = half2_to_float2(codes_to_half2(static_cast<uint16_t>(codes)));
  const float2 b = half2_to_float2(codes_to_half2(static_cast<uint16_t>(codes >> 16)));
  return floats_to_codes(a.x * f, a.y * f) | (floats_to_codes(b.x * f, b.y * f) << 16);
}

// NU: units per thread, ceil(page * Dh / UNIT / AP_THREADS).  Few threads with many units each: what a warp
// spends on finding its page and on the maximum is half of its instructions at 32 elements a lane.
constexpr int AP_THREADS = 128;
template <int NU>
__global__ void __launch_bounds__(AP_THREADS) append_kernel(const AppendParams p) {
  behind_last();
  const Pool& c = p.c;
  const int b = blockIdx.z >> 1, kv = blockIdx.z & 1, h = blockIdx.y;
  const int slot = p.slots[b];
  if (slot == -1) return;                         // a row of padding
  const bool reports = blockIdx.x == 0 && threadIdx.x == 0;
  if (slot < 0 || slot >= c.slots) {
    if (reports) record_pages();
    return;
  }
  const int n = p.n_new ? p.n_new[b] : p.T;
  const int len = c.lens[slot];
  const int p0 = len - n;                         // first new position
  if (n < 0 || n > p.T || p0 < 0 || len > c.max_pages * static_cast<long long>(c.page)) {
    if (reports) record_pages();
    return;
  }
  const int page_shift = 31 - __clz(c.page);
  const int j = (p0 >> page_shift) + blockIdx.x;  // the page's place in the table
  const long long at0 = static_cast<long long>(j) << page_shift;
  if (n == 0 || at0 >= len) return;
  const int pid = c.table[static_cast<long long>(slot) * c.max_pages + j];
  bool bad = pid < 0 || pid >= c.pages;
  if (!bad) bad = c.refs[pid] != 1;               // a page that others hold too is not written
  if (bad) {
    if (threadIdx.x == 0) record_pages();
    return;
  }
  const __nv_bfloat16* src = (kv ? p.v : p.k) + b * (kv ? p.vb : p.kb) + h * (kv ? p.vh : p.kh);
  const long long st = kv ? p.vt : p.kt;
  const long long page_at = (static_cast<long long>(pid) * c.heads + h) * c.page * c.Dh;
  uint8_t* codes = (kv ? c.v : c.k) + page_at;
  float* scale = (kv ? c.v_scale : c.k_scale) + static_cast<long long>(pid) * c.heads + h;
  const int skip = max(0, static_cast<int>(p0 - at0));                       // older tokens in the page
  const int end = static_cast<int>(min(static_cast<long long>(c.page), len - at0));
  const int row_shift = c.Dh == 128 ? 4 : 3;      // units of a row: 16 or 8
  src += (at0 - p0) * st;

  const int t0 = threadIdx.x >> row_shift, t_step = AP_THREADS >> row_shift;   // unit i: token t0 + i * t_step
  const __nv_bfloat16* from = src + t0 * st + (threadIdx.x & ((1 << row_shift) - 1)) * UNIT;
  uint4 x[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int t = t0 + i * t_step;
    x[i] = make_uint4(0, 0, 0, 0);
    if (t >= skip && t < end) x[i] = *reinterpret_cast<const uint4*>(from);
    from += t_step * st;
  }
  const float old_scale = skip ? *scale : 0.f;
  // Two running magnitudes per word; whether anything is not finite shows in the plain maximum, and
  // only then are the finite ones looked for.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NU; ++i)
    for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w})
      top = __vmaxu2(top, w & 0x7fff7fffu);
  uint32_t amax = max(top >> 16, top & 0xffffu);
  if (amax >= BF16_INF) {
    top = 0;
#pragma unroll
    for (int i = 0; i < NU; ++i)
      for (uint32_t w : {x[i].x, x[i].y, x[i].z, x[i].w})
        top = __vmaxu2(top, finite_bits(w));
    amax = max(top >> 16, top & 0xffffu) | 0x10000u;
  }
  const uint32_t flag = __any_sync(0xffffffffu, amax >> 16) ? 0x10000u : 0u;
  __shared__ unsigned s_max[AP_THREADS / 32];
  const unsigned wmax = __reduce_max_sync(0xffffffffu, amax & 0xffffu) | flag;
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = wmax;
  if (named_before(p.slots, b, slot)) {           // barrier: s_max and every read of the old scale
    if (reports) record_pages();
    return;
  }
  unsigned m = 0, odd = 0;
#pragma unroll
  for (int i = 0; i < AP_THREADS / 32; ++i) {
    m = max(m, s_max[i] & 0xffffu);
    odd |= s_max[i] >> 16;
  }
  int e = scale_exponent(__uint_as_float(m << 16));
  int e_old = e;
  if (skip) {
    e_old = min(max(exponent_of(old_scale), E_MIN), E_MAX);
    e = max(e, e_old);
  }
  const float inv = two_to(-e);
  const float shrink = two_to(max(e_old - e, -126));
  const bool exact_range = odd || e == E_MAX;     // the same in the whole block
  uint2* dst = reinterpret_cast<uint2*>(codes) + threadIdx.x;
  auto mine = [&](int i) {
    const int t = t0 + i * t_step;
    return t >= skip && t < end;
  };
  if (exact_range) {
#pragma unroll
    for (int i = 0; i < NU; ++i)
      if (mine(i)) dst[i * AP_THREADS] = quantise8<true>(x[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < NU; ++i)
      if (mine(i)) dst[i * AP_THREADS] = quantise8<false>(x[i], inv);
  }
  if (e > e_old) {                                // restate what the page held before
#pragma unroll 1
    for (int i = 0; i < NU; ++i)
      if (t0 + i * t_step < skip) {
        const uint2 o = dst[i * AP_THREADS];
        dst[i * AP_THREADS] = make_uint2(restate4(o.x, shrink), restate4(o.y, shrink));
      }
  }
  if (threadIdx.x == 0) *scale = two_to(e);
}

struct ReadParams {
  Pool c;                      // one layer
  const int *slots, *start;    // start null: 0
  __nv_bfloat16 *k, *v;        // [B][heads][length][Dh]
  int fill_k, fill_v;          // rows of padding are zeroed; otherwise left alone
  int length;
};

// Positions start .. start + length - 1 of each sequence; zero behind its end (and before 0).  Bound:
// memory, 1 byte in and 2 out per element; a thread moves READ_UNITS units, loads first.
constexpr int READ_UNITS = 4;
template <int HD>
__global__ void __launch_bounds__(IO_THREADS) read_kernel(const ReadParams p) {
  behind_last();
  constexpr int PER_ROW = HD / UNIT;
  const Pool& c = p.c;
  const int b = blockIdx.z >> 1, kv = blockIdx.z & 1, h = blockIdx.y;
  const int slot = p.slots[b];
  const bool held = slot >= 0 && slot < c.slots;
  if (!held) {
    if (slot != -1 && blockIdx.x == 0 && threadIdx.x == 0) record_pages();
    if (!(kv ? p.fill_v : p.fill_k)) return;
  }
  const int start = p.start && held ? p.start[b] : 0;
  int len = held ? c.lens[slot] : 0;
  if (len < 0 || len > c.max_pages * static_cast<long long>(c.page)) {   // holds nothing that could be read
    if (blockIdx.x == 0 && threadIdx.x == 0) record_pages();
    len = 0;
  }
  const int* row = c.table + static_cast<long long>(held ? slot : 0) * c.max_pages;
  const int page_shift = 31 - __clz(c.page);
  const uint8_t* codes = kv ? c.v : c.k;
  const float* scales = kv ? c.v_scale : c.k_scale;
  const int col = (threadIdx.x % PER_ROW) * UNIT;
  const long long t0 = static_cast<long long>(blockIdx.x) * (READ_UNITS * IO_THREADS / PER_ROW) + threadIdx.x / PER_ROW;
  uint2 w[READ_UNITS];
  float s[READ_UNITS];
#pragma unroll
  for (int i = 0; i < READ_UNITS; ++i) {
    const long long t = t0 + i * (IO_THREADS / PER_ROW), pos = start + t;
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (t < p.length && pos >= 0 && pos < len) {
      const int pid = row[pos >> page_shift];
      if (pid < 0 || pid >= c.pages) {
        record_pages();
      } else {
        const long long ph = static_cast<long long>(pid) * c.heads + h;
        w[i] = *reinterpret_cast<const uint2*>(codes + (((ph << page_shift) + (pos & (c.page - 1))) * HD + col));
        s[i] = scales[ph];
      }
    }
  }
  __nv_bfloat16* out = (kv ? p.v : p.k) + (static_cast<long long>(b) * c.heads + h) * p.length * HD + col;
#pragma unroll
  for (int i = 0; i < READ_UNITS; ++i) {
    const long long t = t0 + i * (IO_THREADS / PER_ROW);
    if (t >= p.length) break;
    uint32_t y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t in = k < 2 ? w[i].x : w[i].y;
      const float2 f = half2_to_float2(codes_to_half2(static_cast<uint16_t>(k & 1 ? in >> 16 : in)));
      y[k] = pack_bf16x2(f.x * s[i], f.y * s[i]);
    }
    *reinterpret_cast<uint4*>(out + t * HD) = make_uint4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace cache
}  // namespace ra
