// Host side of the rotary positions: argument checks, the choice of the access width and the
// launch.  Included once, at the end of ring_attn.cu (it uses that file's helpers).
#pragma once
#include "rope.cuh"

namespace {

// Bytes from the first to behind the last element of a [B][H][S][Dh] view.
long long rope_extent(long long sb, long long sh, long long ss, int B, int H, int S, int Dh) {
  return (B - 1) * sb + (H - 1) * sh + (S - 1) * ss + Dh;
}

int rope_tensor(ra::rope::Tensor* t, const void* x, void* y, int H, const long long* st, int B, int S, int Dh,
                int size) {
  if (!x || !y || !st || H <= 0) return RA_ERR_ARG;
  const int n[3] = {B, H, S};
  long long d[6];   // strides, those of dimensions of one element dropped
  for (int i = 0; i < 6; ++i) {
    d[i] = n[i % 3] == 1 ? 0 : st[i];
    if (d[i] < 0 || d[i] > (1ll << 59) / n[i % 3]) return RA_ERR_SHAPE;
  }
  // Every output element is written by one thread: going up the strides, each dimension has to
  // step over all of the smaller ones.
  bool seen[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
  for (long long reach = Dh;;) {
    int m = -1;
    for (int i = 0; i < 3; ++i)
      if (!seen[i] && (m < 0 || d[3 + i] < d[3 + m])) m = i;
    if (m < 0) break;
    if (d[3 + m] < reach) return RA_ERR_SHAPE;
    reach += d[3 + m] * (n[m] - 1);
    seen[m] = true;
  }
  *t = {x, y, d[0], d[1], d[2], d[3], d[4], d[5], H};
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x), ya = reinterpret_cast<uintptr_t>(y);
  if (xa % size || ya % size) return RA_ERR_ALIGN;
  bool same = xa == ya;
  for (int i = 0; i < 3; ++i) same = same && d[i] == d[i + 3];
  const uintptr_t xe = xa + rope_extent(d[0], d[1], d[2], B, H, S, Dh) * size;
  const uintptr_t ye = ya + rope_extent(d[3], d[4], d[5], B, H, S, Dh) * size;
  if (!same && xa < ye && ya < xe) return RA_ERR_ARG;   // in place, or apart
  return RA_OK;
}

// Whether a [B][H][S][Dh] view at `x` (element size `size`, strides st[3]) has an element at address `a`: going down
// the strides, each index as far as it goes (exact where each dimension steps over the smaller ones, as outputs do).
bool rope_has(const void* x, const long long* st, int B, int H, int S, int Dh, int size, uintptr_t a) {
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x);
  if (a < x0) return false;
  long long off = static_cast<long long>((a - x0) / size);
  const int n[3] = {B, H, S};
  bool done[3] = {false, false, false};
  for (int k = 0; k < 3; ++k) {
    int m = -1;
    for (int i = 0; i < 3; ++i)
      if (!done[i] && (m < 0 || st[i] > st[m])) m = i;
    done[m] = true;
    if (st[m] > 0) off -= st[m] * (off / st[m] < n[m] - 1 ? off / st[m] : n[m] - 1);
  }
  return off < Dh;
}

// Whether one of two views has the other's first or last element: rows of one buffer side by side do not.
bool rope_meet(const void* x, const long long* xs, int xh, const void* y, const long long* ys, int yh, int B, int S, int Dh,
               int size) {
  const auto ends = [&](const void* p, const long long* st, int h, uintptr_t* e) {
    e[0] = reinterpret_cast<uintptr_t>(p);
    e[1] = e[0] + (rope_extent(st[0], st[1], st[2], B, h, S, Dh) - 1) * size;
  };
  uintptr_t ex[2], ey[2];
  ends(x, xs, xh, ex);
  ends(y, ys, yh, ey);
  for (int i = 0; i < 2; ++i)
    if (rope_has(x, xs, B, xh, S, Dh, size, ey[i]) || rope_has(y, ys, B, yh, S, Dh, size, ex[i])) return true;
  return false;
}

// One thread a unit of a token, p.units of them a row.
int rope_launch(void (*kernel)(ra::rope::Params), ra::rope::Params& p, int sm_count, cudaStream_t stream) {
  using namespace ra::rope;
  const long long threads = p.tokens * p.units;
  p.wide_ids = threads > UINT_MAX - THREADS;
  const long long blocks = (threads + THREADS - 1) / THREADS;
  const int heads = p.t[0].heads + p.t[1].heads;
  // As many heads per thread (one sine and cosine for all of them) as leave 8 blocks per SM.  Measured
  // (16K prompt / float32 gradient): 4 blocks 53.6 / 15.2 us, 8 49.5 / 15.0, 16 50.9 / 16.3, 32 58.9 / 19.2.
  int hpt = 1;
  while (hpt < heads && hpt < 16 && blocks * ((heads + 2 * hpt - 1) / (2 * hpt)) >= 8ll * sm_count) hpt *= 2;
  p.heads_per_thread = hpt;
  const int gy = (heads + hpt - 1) / hpt;
  if (blocks > INT_MAX || gy > 65535) return RA_ERR_SHAPE;
  kernel<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(gy)), THREADS, 0, stream>>>(p);
  return launch_status();
}

template <typename T, int N, bool VECTOR>
int rope_units(ra::rope::Params& p, int sm_count, bool interleaved, cudaStream_t stream) {
  using namespace ra::rope;
  p.rot_units = interleaved ? p.rot / N : p.rot / 2 / N;
  p.units = p.rot_units + (p.Dh - p.rot) / N;
  if constexpr (N == 2 && !VECTOR) {   // interleaved pairs alone come here
    return rope_launch(rope_kernel<T, N, true, VECTOR>, p, sm_count, stream);
  } else {
    if constexpr (N == 2) {
      if (interleaved) return rope_launch(rope_kernel<T, N, true, VECTOR>, p, sm_count, stream);
    }
    return rope_launch(rope_kernel<T, N, false, VECTOR>, p, sm_count, stream);
  }
}

template <typename T, int N, bool INTERLEAVED>
int rope_rows(ra::rope::Params& p, int sm_count, cudaStream_t stream) {
  p.units = p.Dh / N;
  return rope_launch(ra::rope::rope_rows_kernel<T, N, INTERLEAVED>, p, sm_count, stream);
}

template <typename T>
int rope_dispatch(ra::rope::Params& p, int sm_count, bool interleaved, cudaStream_t stream) {
  constexpr int WIDE = 16 / static_cast<int>(sizeof(T));
  // The widest access that every row start allows,
  auto rows_fit = [&](int m) {
    if (p.Dh % m) return false;
    for (const ra::rope::Tensor& t : p.t) {
      if (!t.heads) continue;
      if (reinterpret_cast<uintptr_t>(t.x) % (m * sizeof(T)) || reinterpret_cast<uintptr_t>(t.y) % (m * sizeof(T)))
        return false;
      for (long long st : {t.xb, t.xh, t.xs, t.yb, t.yh, t.ys})
        if (st % m) return false;
    }
    return true;
  };
  // and the pairs' distance and the untouched rest.
  auto fits = [&](int m) { return (interleaved ? p.rot : p.rot / 2) % m == 0 && (p.Dh - p.rot) % m == 0 && rows_fit(m); };
  if (interleaved) {
    // rope_rows_kernel (float32 gradient 13.2 us, rope_kernel 14.9; bf16, 40 of 64, 64 + 16 heads 43 and 53)
    if constexpr (WIDE == 8) {
      if (rows_fit(8)) return rope_rows<T, 8, true>(p, sm_count, stream);
    }
    if (rows_fit(4)) return rope_rows<T, 4, true>(p, sm_count, stream);
    if (fits(2)) return rope_units<T, 2, true>(p, sm_count, true, stream);
    return rope_units<T, 2, false>(p, sm_count, true, stream);   // a pair is still one thread's: rot and Dh are even
  }
  // Half: rope_kernel where the pairs lie at a vector's distance (the 16K prompt 49 us, rope_rows_kernel 53), else
  // rope_rows_kernel (bf16, 30 of 64, 64 + 16 heads 48 us, rope_kernel 147; 102 of 128, 2 + 2 heads 54 and 94).
  // Vectors of 4 bf16 there: of 8, 52 and 43 us.
  if constexpr (WIDE == 8) {
    if (fits(8)) return rope_units<T, 8, true>(p, sm_count, false, stream);
  }
  if (fits(4)) return rope_units<T, 4, true>(p, sm_count, false, stream);
  const int units = p.Dh / 4;
  if (rows_fit(4) && units <= 32 && 32 % units == 0) return rope_rows<T, 4, false>(p, sm_count, stream);
  if (fits(2)) return rope_units<T, 2, true>(p, sm_count, false, stream);
  return rope_units<T, 1, false>(p, sm_count, false, stream);
}

}  // namespace

extern "C" {

int ring_attn_rope(const void* q, void* q_out, int Hq, const long long* q_strides, const void* k, void* k_out, int Hk,
                   const long long* k_strides, int B, int S, int Dh, const unsigned long long* steps, int rot,
                   int interleaved, float amplitude, const long long* pos, long long pos_stride_b,
                   long long pos_stride_s, long long offset, int inverse, ra_dtype dtype, ra_stream stream) {
  if (!steps || B <= 0 || S <= 0 || Dh <= 0 || !std::isfinite(amplitude)) return RA_ERR_ARG;
  if (dtype != RA_BF16 && dtype != RA_F32) return RA_ERR_ARG;
  if (Dh % 2 || Dh > 1024 || rot <= 0 || rot > Dh || rot % 2) return RA_ERR_SHAPE;
  if (pos && (pos_stride_b < 0 || pos_stride_s < 0)) return RA_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(steps) % 8 || reinterpret_cast<uintptr_t>(pos) % 8) return RA_ERR_ALIGN;
  const int size = dtype == RA_BF16 ? 2 : 4;
  ra::rope::Params p{};
  int st = rope_tensor(&p.t[0], q, q_out, Hq, q_strides, B, S, Dh, size);
  if (st != RA_OK) return st;
  if (k || k_out || Hk) {
    if ((st = rope_tensor(&p.t[1], k, k_out, Hk, k_strides, B, S, Dh, size)) != RA_OK) return st;
    // written by one thread, read or written by another
    const ra::rope::Tensor &a = p.t[0], &b = p.t[1];
    const long long ai[3] = {a.xb, a.xh, a.xs}, ao[3] = {a.yb, a.yh, a.ys}, bi[3] = {b.xb, b.xh, b.xs}, bo[3] = {b.yb, b.yh, b.ys};
    if (rope_meet(a.y, ao, Hq, b.y, bo, Hk, B, S, Dh, size) || rope_meet(a.y, ao, Hq, b.x, bi, Hk, B, S, Dh, size) ||
        rope_meet(a.x, ai, Hq, b.y, bo, Hk, B, S, Dh, size))
      return RA_ERR_ARG;
  }
  if (static_cast<long long>(Hq) + Hk > 65535) return RA_ERR_SHAPE;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  p.steps = steps;
  p.pos = pos;
  p.pos_b = pos_stride_b;
  p.pos_s = pos_stride_s;
  p.offset = offset;
  p.tokens = static_cast<long long>(B) * S;
  p.S = S;
  p.Dh = Dh;
  p.rot = rot;
  p.amplitude = amplitude;
  p.inverse = inverse != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == RA_BF16 ? rope_dispatch<__nv_bfloat16>(p, di->sm_count, interleaved != 0, s)
                          : rope_dispatch<float>(p, di->sm_count, interleaved != 0, s);
}

}  // extern "C"
