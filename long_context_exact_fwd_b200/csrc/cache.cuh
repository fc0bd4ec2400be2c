// The 8-bit key/value cache: what its kernels share.
//
// Pages of `page` tokens hold e4m3 codes of one head's keys (or values), [page][Dh]; a page and
// head has one scale for its keys and one for its values, a power of two 2^e:
//   value = code * 2^e,   e = least e with amax <= 448 * 2^e, within [E_MIN, E_MAX].
// A power of two leaves a value's relative rounding alone (e4m3 is a floating type: only range and
// underflow depend on the scale), makes every dequantised value exact in bf16, and lets a page's
// older codes be restated at a grown scale exactly, but for what falls below e4m3's smallest
// normal.  E_MIN keeps the smallest code * 2^E_MIN a normal float, E_MAX covers bf16's range.
//
// Slots, lengths, tables and page numbers live in device memory, where the host cannot check them:
// every kernel checks what it reads from them before it goes by it, leaves out what is out of
// range and records RA_ERR_PAGES in a status word of the cache's own (a kernel's RA_ERR_TIMEOUT, in g_status, means
// that a result is incomplete, and neither may hide the other).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "ra_sm100.cuh"

namespace ra {
namespace cache {

constexpr int E_MIN = -117, E_MAX = 120;
constexpr int MAX_BATCH = 1024;

struct Pool {                 // one layer's view, or all layers' (page operators)
  uint8_t *k, *v;             // [layers][pages][heads][page][Dh]
  float *k_scale, *v_scale;   // [layers][pages][heads]
  int *table, *lens, *refs;   // [slots][max_pages], [slots], [pages]
  int layers, pages, heads, page, Dh, slots, max_pages;
};

__device__ int g_pages;       // 0, or RA_ERR_PAGES; ring_attn_device_status reads and clears it
__device__ __forceinline__ void record_pages() { atomicExch(&g_pages, RA_ERR_PAGES); }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float scale) { return static_cast<int>((__float_as_uint(scale) >> 23) & 255u) - 127; }

// The scale's exponent for a finite amax >= 0: amax = 1.f * 2^y <= 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, E_MIN), E_MAX);   // amax 0 and subnormals come out below E_MIN
}

// Two e4m3 codes (low byte first) as half2 bits; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// Two floats as e4m3 codes, nearest even, `lo` in the low byte; NaN as NaN.
__device__ __forceinline__ uint32_t floats_to_codes(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// What ran before on the stream is complete; the next launch may be set up from here on.  First in every kernel, on
// every path: a block that ended without waiting would let a later launch pass an unfinished one.
__device__ __forceinline__ void behind_last() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
}

// Whether an earlier entry of the batch names the same slot (the whole block asks; barrier inside).
__device__ __forceinline__ bool named_before(const int* slots, int b, int slot) {
  bool dup = false;
  for (int i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
  return __syncthreads_or(dup) != 0;
}

// The last i in [0, n) with first[i] <= x (first[] is a prefix sum, first[0] = 0).
__device__ __forceinline__ int find_row(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace cache
}  // namespace ra
