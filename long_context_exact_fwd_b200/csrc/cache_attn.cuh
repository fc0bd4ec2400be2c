// Attention of a few new queries per sequence over the 8-bit paged cache.
//
//   s_j = scale * q . k_j over the keys the query sees,  lse = log sum_j exp s_j,
//   o = sum_j exp(s_j - lse) v_j;   a query that sees no key: o = 0, lse = -inf.
//
// The rows of one kv head are its g query heads times the T new tokens (row = t * g + head), taken
// 8 * NT at a time.  Products are computed transposed, S^T = K Q^T and O^T = V^T P^T, with
// mma.sync.m16n8k16: the 16 rows are tokens (then head columns) and the 8 columns are queries, so
// 8 query rows cost one MMA column block and each code is turned into an fp16 fragment once, in
// registers, for all rows.  A token's 128 codes are spread so that a thread's fragments come from
// whole 16-byte words: any order of the contracted index is right if both operands share it.
//
// Numbers.  Codes are exact in fp16.  A query row is scaled by a power of two to just below fp16's
// top and keeps its bf16 values exactly down to 2^-29 of the row's largest; scores and sums are
// fp32.  P carries the value scale 2^e_j of its page, and is rounded to fp16 (half a step, 2^-11 of the term;
// bf16's is 2^-8).  Each row has two references, raised when a term passes one by 2^8: R over its scores
// x_j (log2 units) and R + K, K a whole number, over x_j + e_j:
//   w_j = 2^(x_j + e_j - R - K + 7),   l = sum 2^(K - 7 - e_j) w_j,   o = 2^(K - 7) sum w_j code_j / l,
// so that P's bits go by what a token adds to the row's own result: terms down to 2^-21 of the row's largest
// softmax weight x value scale keep all 11 bits, smaller ones an absolute 2^-32 of it.  (One unit for a warp's rows,
// from the largest scale read, lost rows whose weight lay on pages of small values.)  w_j is taken at no less
// than 2^-93 of 2^(x_j - R), where it is 0 in fp16 and l still has it; the sums use unrounded terms.
//
// Bound: memory, 2 Dh bytes per token and head.  Work is a line of 32-token tiles over (sequence,
// head, row block); every block takes an equal stretch of it, whatever the lengths (they are only
// known on the device), so stretches end inside sequences: such parts go to the workspace and a
// second, small launch joins them.  Each warp streams its own tiles with cp.async through a private
// ring in shared memory, no block barrier inside a stretch (TMA boxes in its place: 7 % slower).
// Measured on B200, 8 heads of 128, 4 query heads each: one context of 512K tokens 170 us, 97 % of a copy's
// rate; 128K 50 us (81 %, some 9 us are start, join and launches); 32 of 16 to 16384 tokens 93 us (89 %).
// The row's own references cost 1 to 2 % at 8 rows, 3 to 10 % at 24 (the unit of a warp's rows: 92 us for the 32).
#pragma once
#include "cache.cuh"

namespace ra {
namespace cache {

constexpr int AT_WARPS = 4;
// Blocks per SM (one joins its warps while the others stream), by the registers that NT and the head take;
// each warp's ring has two stages.  Measured, heads of 128: one context of 512K, 16 rows (NT 2), 2 blocks of 3
// stages 185 us, 3 of 2 180; 24 rows, 3 stages and 2 234 and 232; 32 contexts up to 16K, NT 1, 2 blocks of 3
// stages 98.9, 3 of 2 94.8.  Heads of 64, 16 contexts up to 64K: NT 1, 3 blocks 58.9 and 4 57.6 us; NT 2, 2 87.5,
// 3 76.5 and 4 no better; NT 3, 2 103.8 and 3 94.9.
__host__ __device__ constexpr int at_per_sm(int hd, int nt) { return hd == 64 ? (nt == 1 ? 4 : 3) : (nt == 3 ? 2 : 3); }
constexpr int AT_STAGES = 2;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int AT_TILE = 32;          // tokens of a warp's tile
constexpr int AT_MAX_SMS = 160;      // SMs that the workspace has room for
// What starting and joining a stretch costs, in tiles: it counts in a block's share.  Measured for 32
// contexts of 16 to 16384 tokens, 8 heads: 0 115.8 us, 8 102.2, 16 98.7, 24 100.4.
constexpr int AT_START = 16;
// Tiles of a stretch, at least: one a warp.  Measured (one context of 777 / 8192 tokens): 4 9.1 / 12.0 us,
// 8 10.0 / 12.4, 16 12.1 / 13.7.
constexpr int AT_LEAST = 4;
constexpr float AT_RAISE = 8.f;      // log2: P <= 2^8, times 2^7 still an fp16 number
constexpr float AT_P_LOG2 = 7.f;     // P is held at 2^7 times its value
constexpr float AT_W_LEAST = -93.f;  // log2 of w_j / 2^(x_j - R), at least
constexpr float AT_L_MOST = 9.903520314283042e27f;   // 2^93
constexpr float NOTHING = 3.4028234663852886e38f;   // minus the reference of a row that has seen nothing: any score raises it

struct AttendParams {
  Pool c;                      // one layer
  const __nv_bfloat16* q;      // [B][Hq][T][Dh], strides in elements
  long long qb, qh, qt;
  const int *slots, *n_new;    // n_new null: T
  void* o;                     // [B][Hq][T][Dh] bf16 (or fp32)
  float* lse;                  // [B][Hq][T]
  float* part;                 // [2 * CTAs][8 NT rows][Dh + 4]: O, then m and l
  // What is to be joined: a segment's last and first block, and b, h * n_blocks + row block; last < 0: nothing.
  // By segment ([B * heads * n_blocks]) if there are few, else by the block it starts in ([CTAs]).
  int4* split;
  int by_segment;
  int B, T, g, n_blocks;       // row blocks per (sequence, head)
  int page_shift, causal, o_f32;
  int fill_o, fill_lse;        // rows of padding get o = 0, lse = -inf; otherwise they are left alone
  float scale_log2;
};

template <int HD, int NT>
struct AttLayout {
  static constexpr int STAGES = AT_STAGES;
  static constexpr int KV = AT_TILE * HD;              // bytes of a tile's keys
  static constexpr int STAGE = 2 * KV;
  static constexpr int RING = STAGES * STAGE;          // per warp
  static constexpr int SCALES = AT_WARPS * RING;       // [warp][stage][4] floats
  static constexpr int ML = SCALES + AT_WARPS * STAGES * 16;   // [warp][rows][2] floats, rows <= 32
  static constexpr int NANS = ML + AT_WARPS * 32 * 8;  // [HD] ints
  // [NT][HD / 16][32] uint2, fragments of the queries: shared by the warps, read again for every tile (in
  // registers: 16 rows on 512K tokens 197 us, so 185)
  static constexpr int Q = NANS + HD * 4;
  static constexpr int QS = Q + NT * (HD / 16) * 256;  // [rows] floats, their scales
  static constexpr int PREFIX = QS + 8 * NT * 4;         // [B + 1] ints, then slots, lengths, new tokens [B]
  static int bytes(int B) { return PREFIX + (4 * B + 1) * 4; }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(fill ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  return *reinterpret_cast<const uint4*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  return *reinterpret_cast<const uint2*>(__cvta_shared_to_generic(a));
}
__device__ __forceinline__ void mma_f16(float& c0, float& c1, float& c2, float& c3, const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c0), "+f"(c1), "+f"(c2), "+f"(c3)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ bool has_nan_code(uint32_t w) {
  return (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
}

// Byte offset of 16-byte chunk `chunk` of token `t` in a warp's tile.  Lines of 128 bytes; the
// exclusive-or spreads the eight threads of a shared-memory phase over all banks: keys are read at
// tokens t, t + 1 (four chunks each), values at tokens t, t + 2, t + 4, t + 6 (two chunks each).
template <int HD>
__device__ __forceinline__ uint32_t key_offset(int t, int chunk) {
  return HD == 128 ? t * 128 + ((chunk ^ (t & 1)) << 4) : t * 64 + (chunk << 4);
}
template <int HD>
__device__ __forceinline__ uint32_t value_offset(int t, int chunk) {
  const int line = HD == 128 ? t : t >> 1;
  const int at = HD == 128 ? chunk : ((t & 1) << 2) + chunk;
  return line * 128 + ((at ^ (((t >> 1) & 3) << 1)) << 4);
}

// Four columns of one finished row (row = t * g + head) from its reference m, sum z and average a.
template <int HD>
__device__ __forceinline__ void store_row(const AttendParams& p, int b, int h, int row, int d, float m, float z, float4 a) {
  const int tt = row / p.g, hq = h * p.g + row % p.g;
  const long long at = (static_cast<long long>(b) * p.c.heads * p.g + hq) * p.T + tt;
  if (p.o_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * HD + d) = a;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at * HD + d) =
        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  if (d == 0) p.lse[at] = z == 0.f ? -INFINITY : (m + log2f(z)) * 0.69314718055994531f;
}

// Joins N parts to the average a of reference m and weight z.  Part i: an average y[i] of the values (sums could pass
// float's range where the values are near its end) with its reference and weight ml[i]; weight 0 has seen nothing.  A
// part whose reference lies d <= 0 above the common one counts 2^d, applied in two halves: one of small weight and
// large values may be the result, and 2^d alone ends at 2^-126.  FIRST: a is none yet.
template <bool FIRST, int N>
__device__ __forceinline__ void join_parts(const float2 (&ml)[N], const float4 (&y)[N], float& m, float& z, float4& a) {
  float top = FIRST ? ml[0].x : m;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, ml[i].x);
  auto half_of = [&](float ref) { return ref == top ? 1.f : ex2_approx(0.5f * (ref - top)); };   // nothing yet: weight 0
  const float old = FIRST ? 0.f : half_of(m);
  float half[N], sum = FIRST ? 0.f : z * old * old;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    half[i] = half_of(ml[i].x);
    sum += ml[i].y * half[i] * half[i];
  }
  m = top;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const float w = old * (z * inv);
  a = FIRST ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(a.x * old * w, a.y * old * w, a.z * old * w, a.w * old * w);
  z = sum;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (ml[i].y == 0.f) continue;
    const float h = half[i], x = h * (ml[i].y * inv);
    a = make_float4(fmaf(y[i].x * h, x, a.x), fmaf(y[i].y * h, x, a.y), fmaf(y[i].z * h, x, a.z), fmaf(y[i].w * h, x, a.w));
  }
}

// Rows t >= n[b] (shared memory; 0 for an entry that is left out), 128 tokens of a query head at a time over the grid.
template <int HD>
__device__ __forceinline__ void fill_padding(const AttendParams& p, const int* n) {
  constexpr int AT_ONCE = 128;
  const int heads = p.c.heads * p.g, per_head = (p.T + AT_ONCE - 1) / AT_ONCE;
  const long long units = static_cast<long long>(p.B) * heads * per_head;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long i = u / per_head;                // query head of the whole batch
    const int t = static_cast<int>(u - i * per_head) * AT_ONCE;
    const int t0 = max(t, n[i / heads]), t1 = min(t + AT_ONCE, p.T);
    const long long row = i * p.T + t0;
    if (p.fill_lse)
      for (int k = threadIdx.x; k < t1 - t0; k += blockDim.x) p.lse[row + k] = -INFINITY;
    if (p.fill_o) {
      const int size = p.o_f32 ? 4 : 2;
      uint4* o = reinterpret_cast<uint4*>(static_cast<char*>(p.o) + row * HD * size);
      for (int k = threadIdx.x; k < (t1 - t0) * HD * size / 16; k += blockDim.x) o[k] = make_uint4(0, 0, 0, 0);
    }
  }
}

template <int HD, int NT>
__global__ void __launch_bounds__(AT_THREADS, at_per_sm(HD, NT)) attend_kernel(const AttendParams p) {
  using L = AttLayout<HD, NT>;
  constexpr int ROWS = 8 * NT, STAGES = L::STAGES;
  constexpr int KS = HD / 16;          // k steps of a score, and 16-column blocks of a head
  extern __shared__ __align__(128) uint8_t smem[];
  const Pool& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, gc = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * L::RING;
  uint8_t* ring_ptr = smem + warp * L::RING;
  float* scales = reinterpret_cast<float*>(smem + L::SCALES) + warp * STAGES * 4;
  const uint32_t scales_u = smem_u32(scales);
  float* s_ml = reinterpret_cast<float*>(smem + L::ML);
  int* s_nan = reinterpret_cast<int*>(smem + L::NANS);
  uint2* s_q = reinterpret_cast<uint2*>(smem + L::Q);
  float* s_qs = reinterpret_cast<float*>(smem + L::QS);
  int* s_prefix = reinterpret_cast<int*>(smem + L::PREFIX);
  int *s_slot = s_prefix + p.B + 1, *s_len = s_slot + p.B, *s_n = s_len + p.B;
  __shared__ int s_warp[AT_WARPS];

  asm volatile("griddepcontrol.wait;" ::: "memory");   // what ran before on the stream is complete
  // ---- the line: for each (head, row block) of a sequence AT_START places, then its tiles
  int total = 0;
  bool padding = false;                       // some entry has rows that are none
  for (int b0 = 0; b0 < p.B; b0 += AT_THREADS) {
    const int b = b0 + threadIdx.x;
    int w = 0;
    if (b < p.B) {
      s_n[b] = 0;
      const int slot = p.slots[b];
      if (slot >= 0 && slot < c.slots) {
        const int len = c.lens[slot], n = p.n_new ? p.n_new[b] : p.T;
        const bool ok = n >= 0 && n <= p.T && len >= 0 && len <= c.max_pages * static_cast<long long>(c.page);
        if (!ok && blockIdx.x == 0) record_pages();
        if (ok && n > 0) w = (max(1, (len + AT_TILE - 1) / AT_TILE) + AT_START) * c.heads * p.n_blocks;
        s_slot[b] = slot;
        s_len[b] = len;
        if (ok) s_n[b] = n;
      } else if (slot != -1 && blockIdx.x == 0) {
        record_pages();
      }
      padding |= s_n[b] < p.T;
    }
    if (p.by_segment && blockIdx.x == 0 && b < p.B && w == 0)   // nobody comes by these
      for (int i = 0; i < c.heads * p.n_blocks; ++i) p.split[b * c.heads * p.n_blocks + i] = make_int4(-1, 0, 0, 0);
    // block prefix sum
    int s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += y;
    }
    if (lane == 31) s_warp[warp] = s;
    __syncthreads();
    int before = total, all = total;
#pragma unroll
    for (int i = 0; i < AT_WARPS; ++i) {
      if (i < warp) before += s_warp[i];
      all += s_warp[i];
    }
    if (b < p.B) s_prefix[b] = before + s - w;
    total = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) s_prefix[p.B] = total;
  for (int i = threadIdx.x; i < HD; i += AT_THREADS) s_nan[i] = INT_MAX;
  if (__syncthreads_or(padding && (p.fill_o || p.fill_lse))) fill_padding<HD>(p, s_n);
  const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), AT_LEAST);
  const int line0 = min(static_cast<long long>(total), static_cast<long long>(blockIdx.x) * per);
  const int line1 = min(total, line0 + per);

  asm volatile("griddepcontrol.launch_dependents;");   // the join can take what the SMs have left, and wait
  int4 mine_split = make_int4(-1, 0, 0, 0);
  for (int x = line0; x < line1;) {
    // ---- which sequence, head and row block
    int b = 0;
    {
      int hi = p.B;
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (s_prefix[mid] <= x) b = mid; else hi = mid;
      }
    }
    const int w_b = s_prefix[b + 1] - s_prefix[b];
    const int places = w_b / (c.heads * p.n_blocks), nt = places - AT_START;
    const int seg = (x - s_prefix[b]) / places;
    const int seg0 = s_prefix[b] + seg * places + AT_START;   // of its tiles
    const int h = seg / p.n_blocks, rb = seg - h * p.n_blocks;
    const int t0 = max(0, x - seg0), t1 = min(nt, line1 - seg0);
    x = seg0 + nt;
    if (t0 >= t1) continue;                   // its tiles are the next block's
    const int slot = s_slot[b], len = s_len[b], n = s_n[b];
    const int row0 = rb * ROWS, rows = min(ROWS, n * p.g - row0);
    // keys that a row sees: its token's position + 1 (causal), or all
    auto limit_of = [&](int r) { return p.causal ? max(0, min(len, len - n + (row0 + r) / p.g + 1)) : len; };
    const int lim_min = rows > 0 ? limit_of(0) : 0;
    const int lim_max = rows > 0 ? limit_of(rows - 1) : 0;
    const bool unseen = lim_min < len && t1 * AT_TILE > lim_min;   // tokens here that some row does not see
    const int* table = c.table + static_cast<long long>(slot) * c.max_pages;

    // ---- queries: warp j < NT has rows j * 8 .., lane (gr, gc) row gr's head columns gc * HD / 4 ..; loaded
    // ahead of the page numbers, made fragments behind them
    uint4 raw[KS / 2];
    if (warp < NT) {
      const int r = warp * 8 + gr;
      const int tt = (row0 + r) / p.g, hq = h * p.g + (row0 + r) - tt * p.g;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + b * p.qb + hq * p.qh + tt * p.qt + gc * (HD / 4));
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) raw[i] = r < rows ? src[i] : make_uint4(0, 0, 0, 0);
    }

    // ---- this warp's tiles: t0 + warp, + AT_WARPS, ...; those behind every row's limit are empty
    const int t_end = min(t1, (lim_max + AT_TILE - 1) / AT_TILE);
    const int first = t0 + warp;
    const int count = first < t_end ? (t_end - first + AT_WARPS - 1) / AT_WARPS : 0;
    auto page_of = [&](int tile, int sub) {   // page of the tile's 16-token half `sub`, -1: none
      const int tok = tile * AT_TILE + sub * 16;
      if (tok >= len) return -1;
      const int pid = table[tok >> p.page_shift];
      if (pid < 0 || pid >= c.pages) {
        record_pages();
        return -1;
      }
      return pid;
    };
    int next_pid0 = -1, next_pid1 = -1;
    auto look_up = [&](int i) {
      next_pid0 = next_pid1 = -1;
      if (i < count) {
        const int tile = first + i * AT_WARPS;
        next_pid0 = page_of(tile, 0);
        next_pid1 = p.page_shift == 4 ? page_of(tile, 1) : next_pid0;
      }
    };
    auto fetch = [&](int i) {                 // tile i into its stage; the next one's pages on the way
      if (i < count) {
        const int tile = first + i * AT_WARPS, stage = i % STAGES;
        const int pid0 = next_pid0, pid1 = next_pid1;
        const int in_page = (tile * AT_TILE) & (c.page - 1);
        const long long at0 = ((static_cast<long long>(max(pid0, 0)) * c.heads + h) * c.page + in_page) * HD;
        const long long at1 = p.page_shift == 4
                                  ? (static_cast<long long>(max(pid1, 0)) * c.heads + h) * c.page * HD
                                  : at0 + 16 * HD;
        const uint32_t dst = ring + stage * L::STAGE;
        constexpr int CHUNKS = HD / 16;       // per token
        constexpr int PER_HALF = 16 * CHUNKS / 32;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const long long at = half ? at1 : at0;
          const int pid = half ? pid1 : pid0;
#pragma unroll
          for (int j = 0; j < PER_HALF; ++j) {
            const int ch = j * 32 + lane, t = ch / CHUNKS, k = ch % CHUNKS;
            const int tok = half * 16 + t;
            const bool fill = pid >= 0 && tile * AT_TILE + tok < len;
            cp_async16(dst + key_offset<HD>(tok, k), c.k + at + ch * 16, fill);
            cp_async16(dst + L::KV + value_offset<HD>(tok, k), c.v + at + ch * 16, fill);
          }
        }
        if (lane < 4) {                       // key scales of both halves, then value scales
          const int pid = lane & 1 ? pid1 : pid0;
          const bool fill = pid >= 0 && (!(lane & 1) || tile * AT_TILE + 16 < len);
          cp_async4(scales_u + (stage * 4 + lane) * 4,
                    (lane & 2 ? c.v_scale : c.k_scale) + static_cast<long long>(max(pid, 0)) * c.heads + h, fill);
        }
        look_up(i + 1);
      }
      cp_async_commit();
    };
    look_up(0);
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);

    if (warp < NT) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < KS / 2; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t w = (&raw[i].x)[x];
          const float lo = fabsf(__uint_as_float(w << 16)), hi = fabsf(__uint_as_float(w & 0xffff0000u));
          amax = fmaxf(amax, fmaxf(lo <= 3.4028234663852886e38f ? lo : 0.f, hi <= 3.4028234663852886e38f ? hi : 0.f));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int up = amax > 0.f ? min(max(14 - exponent_of(amax), -113), 126) : 0;   // amax -> [2^14, 2^15)
      const float f = two_to(up);
      auto half2 = [&](uint32_t v) { return pack_half2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f); };
#pragma unroll
      for (int i = 0; i < KS / 2; ++i) {
        s_q[(warp * KS + 2 * i) * 32 + lane] = make_uint2(half2(raw[i].x), half2(raw[i].y));
        s_q[(warp * KS + 2 * i + 1) * 32 + lane] = make_uint2(half2(raw[i].z), half2(raw[i].w));
      }
      if (gc == 0) s_qs[warp * 8 + gr] = p.scale_log2 * two_to(-up);
    }
    __syncthreads();
    float2 row_scale[NT];                     // of the accumulator's columns 2 gc, 2 gc + 1
    int limit[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = j * 8 + 2 * gc + e;
        (e ? row_scale[j].y : row_scale[j].x) = s_qs[rr];
        limit[j][e] = rr < rows ? limit_of(rr) : len;
      }

    float o[KS][NT][4];
    // of columns 2 gc, 2 gc + 1: minus R, minus (R + K), the sum, and 2^(K - 7), the unit of O
    float2 neg_ref[NT], neg_top[NT], l[NT], unit[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      neg_ref[j] = neg_top[j] = make_float2(NOTHING, NOTHING);
      unit[j] = make_float2(two_to(-7), two_to(-7));
      l[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < KS; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[m][j][i] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      fetch(i + STAGES - 1);
      const int tile = first + i * AT_WARPS, stage = i % STAGES, tok0 = tile * AT_TILE;
      const uint32_t kst = ring + stage * L::STAGE, vst = kst + L::KV;
      const float4 sc = *reinterpret_cast<const float4*>(scales + stage * 4);

      // scores: S^T, rows tokens gr and gr + 8 of each half, columns queries 2 gc, 2 gc + 1
      float2 s[2][NT][2];                     // [half][..][token gr or gr + 8]
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < NT; ++j) s[half][j][0] = s[half][j][1] = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < KS / 4; ++w) {      // codes of tokens gr, gr + 8 of both halves: head columns gc * HD / 4 ..
        uint4 k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) k[i] = lds128(kst + key_offset<HD>(i * 8 + gr, gc * (KS / 4) + w));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint2 q[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) q[j] = s_q[(j * KS + 4 * w + x) * 32 + lane];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t lo = (&k[2 * half].x)[x], hi = (&k[2 * half + 1].x)[x];
            const uint32_t a[4] = {codes_to_half2(static_cast<uint16_t>(lo)), codes_to_half2(static_cast<uint16_t>(hi)),
                                   codes_to_half2(static_cast<uint16_t>(lo >> 16)),
                                   codes_to_half2(static_cast<uint16_t>(hi >> 16))};
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma_f16(s[half][j][0].x, s[half][j][0].y, s[half][j][1].x, s[half][j][1].y, a, q[j].x, q[j].y);
          }
        }
      }

      // log2 units, mask, and the largest of each column
      const bool none0 = sc.x == 0.f, none1 = sc.y == 0.f;   // a half without a page (or behind the end) has no scale
      const bool masked = tok0 + AT_TILE > lim_min || none0 || none1;
      const int e0 = exponent_of(sc.z), e1 = exponent_of(sc.w);   // of the halves' value scales
      const float2 up0 = make_float2(e0, e0), up1 = make_float2(e1, e1);
      float top = -INFINITY;                  // over a reference
      float2 mx[NT], my[NT];                  // largest score, and largest with its value scale
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float k = half ? sc.y : sc.x;
          const float2 f = __fmul2_rn(row_scale[j], make_float2(k, k));
#pragma unroll
          for (int y = 0; y < 2; ++y) s[half][j][y] = __fmul2_rn(s[half][j][y], f);
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {       // tokens of the tile, from this thread's first, that are seen
            const bool none = i >> 1 ? none1 : none0;
            if (none || limit[j][0] - tok0 - gr <= 8 * i) s[i >> 1][j][i & 1].x = -INFINITY;
            if (none || limit[j][1] - tok0 - gr <= 8 * i) s[i >> 1][j][i & 1].y = -INFINITY;
          }
        }
        const float2 m0 = make_float2(fmaxf(s[0][j][0].x, s[0][j][1].x), fmaxf(s[0][j][0].y, s[0][j][1].y));
        const float2 m1 = make_float2(fmaxf(s[1][j][0].x, s[1][j][1].x), fmaxf(s[1][j][0].y, s[1][j][1].y));
        const float2 y0 = __fadd2_rn(m0, up0), y1 = __fadd2_rn(m1, up1);
        mx[j] = make_float2(fmaxf(m0.x, m1.x), fmaxf(m0.y, m1.y));
        my[j] = make_float2(fmaxf(y0.x, y1.x), fmaxf(y0.y, y1.y));
        const float2 over = __fadd2_rn(mx[j], neg_ref[j]), over_y = __fadd2_rn(my[j], neg_top[j]);
        top = fmaxf(fmaxf(top, fmaxf(over.x, over.y)), fmaxf(over_y.x, over_y.y));
      }
      if (__any_sync(0xffffffffu, top > AT_RAISE)) {
        auto largest = [](float m) {
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        };
        // returns what O has to be multiplied by
        auto raised = [&](float& ref, float& ref_top, float& sum, float& u, float m, float y) {
          m = largest(fmaxf(-ref, m));
          y = largest(fmaxf(-ref_top, y));
          // never above the largest; both references still at NOTHING: 0
          const float k = fminf(fmaxf(floorf(y - m), E_MIN), E_MAX);
          const float a = -ref - m, f = -ref_top - (m + k);
          sum *= a == 0.f ? 1.f : ex2_approx(a);
          ref = -m;
          ref_top = -(m + k);
          u = two_to(static_cast<int>(k) - 7);
          return f == 0.f ? 1.f : ex2_approx(f);
        };
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float f0 = raised(neg_ref[j].x, neg_top[j].x, l[j].x, unit[j].x, mx[j].x, my[j].x);
          const float f1 = raised(neg_ref[j].y, neg_top[j].y, l[j].y, unit[j].y, mx[j].y, my[j].y);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            o[k][j][0] *= f0;
            o[k][j][1] *= f1;
            o[k][j][2] *= f0;
            o[k][j][3] *= f1;
          }
        }
      }

      // P^T as B fragments
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int e = half ? e1 : e0;
        const float up = static_cast<float>(e) + AT_P_LOG2, inv = two_to(-e);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float2 least = __fadd2_rn(neg_ref[j], make_float2(AT_W_LEAST, AT_W_LEAST));
          float2 at = __fadd2_rn(neg_top[j], make_float2(up, up));
          at = make_float2(fmaxf(at.x, least.x), fmaxf(at.y, least.y));
          float2 back = __fmul2_rn(unit[j], make_float2(inv, inv));
          back = make_float2(fminf(back.x, AT_L_MOST), fminf(back.y, AT_L_MOST));
          float2 w[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 x = __fadd2_rn(s[half][j][y], at);
            w[y] = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            pf[half][j][y] = transpose8(pack_half2(w[y].x, w[y].y));
          }
          l[j] = __ffma2_rn(__fadd2_rn(w[0], w[1]), back, l[j]);
        }
      }

      // O^T += V^T P^T: thread's tokens 2 gc, 2 gc + 1, 2 gc + 8, 2 gc + 9, head columns gr * HD / 8 ..
      // A NaN that some rows of the block do not see must not reach them through 0 * NaN: it is taken out of
      // such tiles, and put back into the rows that see it at the end.
      if (masked && unseen) {
#pragma unroll 1
        for (int i = lane; i < AT_TILE * (HD / 16); i += 32) {
          const int t = i / (HD / 16), chunk = i % (HD / 16);
          uint32_t* at = reinterpret_cast<uint32_t*>(ring_ptr + stage * L::STAGE + L::KV + value_offset<HD>(t, chunk));
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            uint32_t x = at[w];
            if (!has_nan_code(x)) continue;
#pragma unroll 1
            for (int y = 0; y < 4; ++y)
              if (((x >> (8 * y)) & 0x7fu) == 0x7fu) {
                atomicMin(s_nan + chunk * 16 + 4 * w + y, tok0 + t);
                x &= ~(0xffu << (8 * y));
              }
            at[w] = x;
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[4][HD / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = half * 16 + 2 * gc + (k & 1) + (k & 2) * 4;
          if (HD == 128) {
            const uint4 a = lds128(vst + value_offset<HD>(t, gr));
            v[k][0] = a.x; v[k][1] = a.y; v[k][2 % (HD / 32)] = a.z; v[k][3 % (HD / 32)] = a.w;
          } else {
            const uint2 a = lds64(vst + value_offset<HD>(t, gr >> 1) + (gr & 1) * 8);
            v[k][0] = a.x; v[k][1] = a.y;
          }
        }
#pragma unroll
        for (int w = 0; w < HD / 32; ++w) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t lo = __byte_perm(v[0][w], v[1][w], y ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(v[2][w], v[3][w], y ? 0x7362 : 0x5140);
            const uint32_t a[4] = {codes_to_half2(static_cast<uint16_t>(lo)), codes_to_half2(static_cast<uint16_t>(lo >> 16)),
                                   codes_to_half2(static_cast<uint16_t>(hi)), codes_to_half2(static_cast<uint16_t>(hi >> 16))};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float (&c)[4] = o[2 * w + y][j];
              mma_f16(c[0], c[1], c[2], c[3], a, pf[half][j][0], pf[half][j][1]);
            }
          }
        }
      }
    }

    // ---- join the warps: each leaves m, l and its average of the values where its ring was
    cp_async_wait<0>();
    __syncwarp();
    float* mine = reinterpret_cast<float*>(ring_ptr);   // [ROWS][HD]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float z = e ? l[j].y : l[j].x;
        z += __shfl_xor_sync(0xffffffffu, z, 4);
        z += __shfl_xor_sync(0xffffffffu, z, 8);
        z += __shfl_xor_sync(0xffffffffu, z, 16);
        const int r = j * 8 + 2 * gc + e;
        const float u = e ? unit[j].y : unit[j].x, inv = 1.f / z;   // a warp that saw nothing is passed over
        if (gr == 0) {
          s_ml[(warp * 32 + r) * 2] = z == 0.f ? -INFINITY : -(e ? neg_ref[j].y : neg_ref[j].x);
          s_ml[(warp * 32 + r) * 2 + 1] = z;
        }
#pragma unroll
        for (int k = 0; k < KS / 2; ++k)
          *reinterpret_cast<float4*>(mine + r * HD + gr * (HD / 8) + 4 * k) =
              make_float4(o[2 * k][j][e] * inv * u, o[2 * k][j][e + 2] * inv * u, o[2 * k + 1][j][e] * inv * u,
                          o[2 * k + 1][j][e + 2] * inv * u);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
    const int c0 = seg0 / per, c1 = (seg0 + nt - 1) / per;
    constexpr int GROUPS = HD / 4;            // float4 groups of a row
    float* part = p.part + static_cast<long long>(2 * blockIdx.x + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * ROWS * (HD + 4);
    for (int i = threadIdx.x; i < ROWS * GROUPS; i += AT_THREADS) {
      const int r = i / GROUPS, d = (i % GROUPS) * 4;
      if (r >= rows) continue;
      float m, z;
      float4 a;
      float2 ml[AT_WARPS];
      float4 y[AT_WARPS];
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        ml[w] = *reinterpret_cast<const float2*>(s_ml + (w * 32 + r) * 2);
        y[w] = *reinterpret_cast<const float4*>(smem + w * L::RING + (r * HD + d) * 4);
      }
      join_parts<true>(ml, y, m, z, a);
      if (unseen) {
        const int lim = limit_of(r);
        const float nan = __uint_as_float(0x7fffffffu);
        if (s_nan[d] < lim) a.x = nan;
        if (s_nan[d + 1] < lim) a.y = nan;
        if (s_nan[d + 2] < lim) a.z = nan;
        if (s_nan[d + 3] < lim) a.w = nan;
      }
      if (whole) {
        store_row<HD>(p, b, h, row0 + r, d, m, z, a);
      } else {
        float* row = part + r * (HD + 4);
        *reinterpret_cast<float4*>(row + d) = a;
        if (d == 0) *reinterpret_cast<float2*>(row + HD) = make_float2(m, z);
      }
    }
    if (static_cast<int>(blockIdx.x) == c0) {
      const int4 joined = make_int4(whole ? -1 : c1, c0, b, seg);
      if (!p.by_segment) mine_split = joined;   // a segment that ends here does not hide one that does not: it comes first
      else if (threadIdx.x == 0) p.split[b * c.heads * p.n_blocks + seg] = joined;
    }
    __syncthreads();                          // rings and s_nan are free again
    if (unseen) {
      for (int i = threadIdx.x; i < HD; i += AT_THREADS) s_nan[i] = INT_MAX;
      __syncthreads();
    }
  }
  if (!p.by_segment && threadIdx.x == 0) p.split[blockIdx.x] = mine_split;
}

// Joins the parts of the segments that the kernel before left split: block (i, j) has rows LOT j .. of the
// i-th entry's segment, WARPS warps a row, each lane 4 columns of every WARPS-th part.  Parts
// are added in an order that only the lengths fix.  Bound: latency of three dependent reads; one block
// alone doing this at the end of its stretch cost 0.6 us per part.
template <int HD, int ROWS, int LOT, int WARPS>
__global__ void __launch_bounds__(LOT * WARPS * 32) join_kernel(const AttendParams p) {
  constexpr int GROUPS = HD / 4;
  __shared__ float4 s_o[LOT][WARPS][GROUPS];
  __shared__ float2 s_ml[LOT][WARPS];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts are complete
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 d = p.split[blockIdx.x];
  if (d.x < 0) return;
  const int c1 = d.x, c0 = d.y, b = d.z, h = d.w / p.n_blocks;
  const int row0 = (d.w - h * p.n_blocks) * ROWS, rows = min(ROWS, (p.n_new ? p.n_new[b] : p.T) * p.g - row0);
  const int rr = warp / WARPS, w = warp % WARPS;
  const int r = blockIdx.y * LOT + rr;
  const long long step = 2ll * ROWS * (HD + 4);
  // part of block c0: its second place; of a block behind it: the first
  const float* second = p.part + (2ll * c0 + 1) * ROWS * (HD + 4) + r * (HD + 4);
  const float* firsts = p.part + 2ll * c0 * ROWS * (HD + 4) + r * (HD + 4);
  auto part = [&](int k) { return k == 0 ? second : firsts + k * step; };
  const int n = c1 - c0 + 1;
  float m = -INFINITY, z = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int AT_ONCE = WARPS >= 16 ? 16 : 8;   // parts read together, statistics and all
  for (int k0 = w; k0 < n; k0 += AT_ONCE * WARPS) {
    float2 ml[AT_ONCE];
    float4 y[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int k = k0 + i * WARPS;
      ml[i] = make_float2(-INFINITY, 0.f);
      if (k < n) {
        ml[i] = *reinterpret_cast<const float2*>(part(k) + HD);
        if (lane < GROUPS) y[i] = *reinterpret_cast<const float4*>(part(k) + 4 * lane);
      }
    }
    join_parts<false>(ml, y, m, z, a);
  }
  if (lane < GROUPS) s_o[rr][w][lane] = a;
  if (lane == 0) s_ml[rr][w] = make_float2(m, z);
  __syncthreads();
  if (w || lane >= GROUPS || r >= rows) return;
  float2 ml[WARPS];
  float4 y[WARPS];
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    ml[i] = s_ml[rr][i];
    y[i] = s_o[rr][i][lane];
  }
  join_parts<true>(ml, y, m, z, a);
  store_row<HD>(p, b, h, row0 + r, 4 * lane, m, z, a);
}

}  // namespace cache
}  // namespace ra
