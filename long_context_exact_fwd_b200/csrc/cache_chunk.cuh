// Attention of many new queries per sequence (a chunk of a prompt) over the 8-bit paged cache.
//
// Same result as attend_kernel (cache_attn.cuh), for row counts where the products bound: both run
// on tcgen05 with accumulators in tensor memory, as in fwd_kernel (fwd_sm100.cuh), whose issue order
// and softmax this keeps:
//   O0 += P0(j-1) V(j-1);  S0 = Q0 K(j)^T;  O1 += P1(j-1) V(j-1);  S1 = Q1 K(j)^T.
// An item is 256 rows of one kv head (row = t * g + head): two 128-row tiles.  Roles of the 12 warps:
//   0-3, 4-7  softmax of tile 0 and 1 (thread = row = TMEM lane); before it, the row's query to fp16,
//   8         tensor memory and the MMA issue (one thread),
//   9         fetches codes by bulk copies into a stage as soon as it is free,
//   10, 11    convert the codes to the stage's fp16 tile, in place.
// The operands are fp16: codes are exact in it (one conversion instruction per two; as bf16 the
// scale would have to be multiplied in), a query row is scaled to its range by a power of two.
// The scales never touch the tiles: a page's key scale multiplies its 16-column groups of scores, and
// its value scale 2^e_j goes into P with the row's two references, R and R + K, as in attend_kernel:
//   w_j = 2^(x_j - R + max(e_j + 7 - K, -93)),   l += min(2^(K - 7 - e_j), 2^93) w_j,   o = 2^(K - 7) O / l.
// Work is cut as in attend_kernel: one line of 128-key tiles over all items, equal stretches, parts
// joined by chunk_join_kernel.
// Bound: the products, and shared memory, which both operands of S, the tiles of V and the conversion go
// through (about 320 KB a key tile; a tile takes some 4300 cycles, 2048 of them its products).  Measured on
// B200, 16 query heads on 4 of 128, 2048 new tokens: at 16K tokens 292 us, 882 TFLOP/s; at 32K 562 us, 948.
#pragma once
#include "cache_attn.cuh"
#include "cache_io.cuh"

namespace ra {
namespace cache {

constexpr int CH_BM = 128, CH_BN = 128, CH_ROWS = 256, CH_STAGES = 4;
constexpr int CH_THREADS = 384;
constexpr int CH_WARP_MMA = 8, CH_WARP_FETCH = 9, CH_WARP_CONV = 10, CH_CONV_WARPS = 2;
constexpr uint32_t CH_REGS_LAUNCH = 168, CH_REGS_SOFTMAX = 208, CH_REGS_OTHER = 88;
static_assert(2 * (CH_REGS_SOFTMAX - CH_REGS_LAUNCH) <= CH_REGS_LAUNCH - CH_REGS_OTHER, "register split exceeds the pool");
constexpr int CH_MAX_CTAS = 160;      // blocks that the workspace has room for (one per SM)
constexpr int CH_START = 3;          // what starting and ending an item costs, in tiles
constexpr int CH_LEAST = 4;          // tiles of a stretch, at least

// Scale constants of one key tile: lots of 16 keys.
struct alignas(16) ChScales {
  // key scale; e + 7, 2^e the value scale; 2^-e; the least of e + 7 - K.  A lot without a page has no weight and no
  // part in the largest: NaN, -inf, any, -inf.
  float4 lot[8];
  unsigned lots;     // of the tile's eight, those that have a page
};

template <int HD>
struct ChLayout {
  static constexpr int SUB = HD / 64;
  static constexpr int SUB_BYTES = 128 * 128;
  static constexpr int TILE_BYTES = SUB * SUB_BYTES;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TILE_BYTES;
  static constexpr int RAW_OFF = KV_OFF + CH_STAGES * TILE_BYTES;
  static constexpr int BAR_OFF = RAW_OFF + (HD == 128 ? 0 : CH_STAGES * CH_BN * HD);
  static constexpr int B_Q_FULL = 0, B_Q_EMPTY = 1, B_KV_FULL = 2, B_KV_EMPTY = B_KV_FULL + CH_STAGES,
                       B_RAW = B_KV_EMPTY + CH_STAGES, B_S_FULL = B_RAW + CH_STAGES, B_P_READY = B_S_FULL + 2, B_O_FINAL = B_P_READY + 2,
                       B_DRAIN = B_O_FINAL + 2, NUM_BARS = B_DRAIN + 1;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;        // TMEM base, abort flag
  static constexpr int SCALE_OFF = (MISC_OFF + 8 + 15) / 16 * 16;
  static constexpr int NAN_OFF = SCALE_OFF + 4 * sizeof(ChScales);              // [3][8 warps][HD + 4] ints, HD a flag
  static constexpr int BATCH_OFF = NAN_OFF + 3 * 8 * (HD + 4) * 4;      // prefix [B + 1], slot, len, n [B]
  static int bytes(int B) { return BATCH_OFF + (4 * B + 1) * 4 + 1024; }
  // Where a stage's codes arrive: the second half of the stage, which is where the same tokens' second
  // 64-column block goes (HD 128); a place of their own (HD 64, where a stage has room for both).
  __host__ __device__ static constexpr int raw(int stage) {
    return HD == 128 ? KV_OFF + stage * TILE_BYTES + TILE_BYTES / 2 : RAW_OFF + stage * (CH_BN * HD);
  }
  __host__ __device__ static constexpr uint32_t s_col(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + uint32_t(HD) * t; }
};

// fp16 x fp16 -> fp32 (formats 0), otherwise as idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn_major, int b_mn_major) {
  return (1u << 4) | (uint32_t(a_mn_major) << 15) | (uint32_t(b_mn_major) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

// The line of work as every role walks it: items (b, h, i) in order, each CH_START places and then
// its key tiles; a block has places [line0, line1).
struct ChWalk {
  const AttendParams* p;
  const int* batch;            // shared memory: prefix [B + 1], slots, lengths, new tokens [B]
  int b, h, i;                 // the current item
  int first;                   // place of its first tile
  int x, line1;
  int nt, t0, t1;              // its tiles, and this block's [t0, t1)

  __device__ __forceinline__ int slot() const { return batch[p->B + 1 + b]; }
  __device__ __forceinline__ int len() const { return batch[2 * p->B + 1 + b]; }
  __device__ __forceinline__ int n() const { return batch[3 * p->B + 1 + b]; }
  // keys that row r (of the sequence) sees
  __device__ __forceinline__ int limit(int r) const {
    const int l = len();
    return p->causal ? max(0, min(l, l - n() + r / p->g + 1)) : l;
  }
  __device__ __forceinline__ static int tiles(int len, int n, int g, int causal, int i) {
    const int last = min((i + 1) * CH_ROWS, n * g) - 1;
    const int lim = causal ? max(0, min(len, len - n + last / g + 1)) : len;
    return max(1, (lim + CH_BN - 1) / CH_BN);
  }
  __device__ __forceinline__ void here() {
    nt = tiles(len(), n(), p->g, p->causal, i);
    t0 = max(0, x - first);
    t1 = min(nt, line1 - first);
  }
  // Goes on to this block's next piece (the first call: the one it stands on); false at the end.
  __device__ __forceinline__ bool next(bool begin) {
    if (!begin) step();
    for (;;) {
      if (x >= line1) return false;
      here();
      if (t0 < t1) return true;
      step();
    }
  }
  __device__ __forceinline__ void step() {
    x = first + nt;
    first = x + CH_START;
    if (++i * CH_ROWS >= n() * p->g) {
      i = 0;
      if (++h == p->c.heads) {
        h = 0;
        do ++b;
        while (b < p->B && n() == 0);
        if (b == p->B) x = line1;   // behind the last item
      }
    }
  }
};

// ------------------------------------------------------------------ fetching (1 warp)
// Page of each 16-token lot of a key tile, in lanes 0-7 (and again in 8-15 ..); -1: none.
__device__ __forceinline__ int ch_pages(const AttendParams& p, const int* table, int len, int tile) {
  const int tok = tile * CH_BN + (threadIdx.x & 7) * 16;
  if (tok >= len) return -1;
  const int pid = table[tok >> p.page_shift];
  if (pid >= 0 && pid < p.c.pages) return pid;
  record_pages();
  return -1;
}

// Codes of every key and value tile into the upper half of its stage, a bulk copy per 16 tokens, and
// the tile's scale constants.
template <int HD>
__device__ void ch_fetch(const AttendParams& p, ChWalk w, uint8_t* smem, uint32_t sbase, volatile int* abort_flag) {
  using L = ChLayout<HD>;
  const Pool& c = p.c;
  const int lane = threadIdx.x & 31;
  const uint32_t bars = sbase + L::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * i; };
  constexpr uint32_t LOT = 16 * HD;                      // bytes of 16 tokens' codes
  int stage = 0, scale_slot = 0;
  uint32_t phase = 0, armed = 0, armed_parity = 0;       // per stage: ever armed, parity of the last time
  ChScales* scales = reinterpret_cast<ChScales*>(smem + L::SCALE_OFF);
  bool ok = true;
  for (bool go = w.next(true); go && ok; go = w.next(false)) {
    const int len = w.len(), h = w.h;
    const int* table = c.table + static_cast<long long>(w.slot()) * c.max_pages;
    int pid = ch_pages(p, table, len, w.t0);
    for (int tile = w.t0; tile < w.t1 && ok; ++tile) {
      float sk = 0.f;
      int e = 0;
      if (pid >= 0) {
        sk = c.k_scale[static_cast<long long>(pid) * c.heads + h];
        e = exponent_of(c.v_scale[static_cast<long long>(pid) * c.heads + h]);
      }
      const int pid_next = tile + 1 < w.t1 ? ch_pages(p, table, len, tile + 1) : -1;
      const unsigned lots = __ballot_sync(0xffffffffu, pid >= 0) & 0xffu;
      const uint32_t bytes = __popc(lots) * LOT;
      const long long at = ((static_cast<long long>(max(pid, 0)) * c.heads + h) * c.page +
                            ((tile * CH_BN + (lane & 7) * 16) & (c.page - 1))) * HD;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(L::B_KV_EMPTY + stage), phase ^ 1u, abort_flag));
        if (!ok) break;
        if (kv == 0) {                                   // before this tile's keys can be multiplied
          ChScales* s = scales + scale_slot;
          if (lane < 8)
            s->lot[lane] = pid >= 0 ? make_float4(sk, static_cast<float>(e) + AT_P_LOG2, two_to(-e), AT_W_LEAST)
                                    : make_float4(__int_as_float(0x7fffffff), -INFINITY, 0.f, -INFINITY);
          if (lane == 0) s->lots = lots;
          scale_slot = (scale_slot + 1) & 3;
          __syncwarp();
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(L::B_RAW + stage), bytes);   // releases the constants, too
        __syncwarp();
        if (lane < 8 && pid >= 0)
          bulk_load(sbase + L::raw(stage) + lane * LOT, (kv ? c.v : c.k) + at, LOT,
                    bar(L::B_RAW + stage));
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == CH_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      pid = pid_next;
    }
  }
  // the copies land before the block can end (they have, unless a wait gave up)
  for (int i = 0; i < CH_STAGES; ++i)
    if (armed >> i & 1u) drain_wait(bar(L::B_RAW + i), armed_parity >> i & 1u);
}

// ------------------------------------------------------------------ converting (2 warps)
template <int HD>
__device__ void ch_convert(const AttendParams& p, ChWalk w, uint8_t* smem, uint32_t sbase, volatile int* abort_flag) {
  using L = ChLayout<HD>;
  const Pool& c = p.c;
  const int lane = threadIdx.x & 31, cw = (threadIdx.x >> 5) - CH_WARP_CONV;
  const uint32_t bars = sbase + L::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * i; };
  const ChScales* scales = reinterpret_cast<const ChScales*>(smem + L::SCALE_OFF);
  int stage = 0, scale_slot = 0, piece = 0;
  uint32_t phase = 0;
  for (bool go = w.next(true); go; go = w.next(false), piece = piece == 2 ? 0 : piece + 1) {
    const int len = w.len(), h = w.h;
    const int row0 = w.i * CH_ROWS;
    const int* table = c.table + static_cast<long long>(w.slot()) * c.max_pages;
    const int lim_min = w.limit(row0);

    // ---- K and V tiles: HD / 16 lanes a token, 16 codes a lane, AT_ONCE tokens a warp step
    constexpr int LANES = HD / 16, AT_ONCE = 32 / LANES, STEPS = CH_BN / (AT_ONCE * CH_CONV_WARPS);
    // HD 128: half a warp has the tokens' first 64 columns, the other half their second
    const int sub = HD == 128 ? lane >> 4 : 0, tok = cw * AT_ONCE + ((lane >> 2) & (AT_ONCE - 1)), c4 = lane & 3;
    const int col = sub * 4 + c4;
    // Token t's row of a 64-column block lies at t * 128, its 16-byte chunks exchanged by t & 7: the eight
    // threads of a phase (two tokens, four lanes each) meet all banks.
    const int at0 = ((2 * c4) ^ (tok & 7)) << 4, at1 = ((2 * c4 + 1) ^ (tok & 7)) << 4;
    static_assert(AT_ONCE * CH_CONV_WARPS % 8 == 0, "a lane's tokens share their place in the swizzle");
    for (int tile = w.t0; tile < w.t1; ++tile) {
      const int tok0 = tile * CH_BN;
      const bool diagonal = lim_min < len && tok0 + CH_BN > lim_min;   // some row does not see all
      unsigned lots = 0;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::B_RAW + stage), phase, abort_flag))) return;
        if (kv == 0) lots = scales[scale_slot].lots;
        const bool plain = lots == 0xffu && tok0 + CH_BN <= len && !diagonal;
        const uint8_t* raw = smem + L::raw(stage) + tok * HD + col * 16;
        uint8_t* dst = smem + L::KV_OFF + stage * L::TILE_BYTES + sub * L::SUB_BYTES + tok * 128;
        bool odd = false;
        // Short: this loop and the softmax's share the instruction cache.  Unrolled over the tile, every role
        // ran at less than half its speed; 2048 queries on 16K tokens, 1, 2, 4 and 8 loads together: 332, 285,
        // 293 and 309 us.
#pragma unroll 1
        for (int k0 = 0; k0 < STEPS; k0 += 2) {
          uint4 x[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(raw + (k0 + k) * (AT_ONCE * CH_CONV_WARPS) * HD);
          __syncwarp();   // HD 128: a token's second block is written where its codes were
          if (!plain) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = tok + (k0 + k) * (AT_ONCE * CH_CONV_WARPS);
              // what lies behind the end, or was not fetched, is 0
              if (!(lots >> (t >> 4) & 1u) || tok0 + t >= len) x[k] = make_uint4(0, 0, 0, 0);
              odd |= kv && diagonal &&
                     (has_nan_code(x[k].x) || has_nan_code(x[k].y) || has_nan_code(x[k].z) || has_nan_code(x[k].w));
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint4 lo = make_uint4(
                codes_to_half2(static_cast<uint16_t>(x[k].x)), codes_to_half2(static_cast<uint16_t>(x[k].x >> 16)),
                codes_to_half2(static_cast<uint16_t>(x[k].y)), codes_to_half2(static_cast<uint16_t>(x[k].y >> 16)));
            const uint4 hi = make_uint4(
                codes_to_half2(static_cast<uint16_t>(x[k].z)), codes_to_half2(static_cast<uint16_t>(x[k].z >> 16)),
                codes_to_half2(static_cast<uint16_t>(x[k].w)), codes_to_half2(static_cast<uint16_t>(x[k].w >> 16)));
            uint8_t* row = dst + (k0 + k) * (AT_ONCE * CH_CONV_WARPS) * 128;
            *reinterpret_cast<uint4*>(row + at0) = lo;
            *reinterpret_cast<uint4*>(row + at1) = hi;
          }
        }
        // A NaN among values that some rows of the item do not see must not reach them through 0 * NaN:
        // it becomes 0 in the tile, and is put back into the rows that see it at the end.
        if (odd) {
#pragma unroll 1
          for (int k = 0; k < STEPS; ++k) {
            const int t_in = tok + k * (AT_ONCE * CH_CONV_WARPS), t = tok0 + t_in;
            if (t >= len) continue;
            const int pg = table[t >> p.page_shift];
            if (pg < 0 || pg >= c.pages) continue;
            const uint8_t* codes = c.v + ((static_cast<long long>(pg) * c.heads + h) * c.page + (t & (c.page - 1))) * HD + col * 16;
#pragma unroll 1
            for (int z = 0; z < 16; ++z) {
              if ((codes[z] & 0x7fu) != 0x7fu) continue;
              const int chunk = (2 * c4 + (z >> 3)) ^ (tok & 7);
              *reinterpret_cast<uint16_t*>(dst + k * (AT_ONCE * CH_CONV_WARPS) * 128 + (chunk << 4) + (z & 7) * 2) = 0;
#pragma unroll 1
              for (int sw = 0; sw < 8; ++sw) {           // each softmax warp has its own list, and clears it
                int* nans = reinterpret_cast<int*>(smem + L::NAN_OFF) + (piece * 8 + sw) * (HD + 4);
                atomicMin(nans + col * 16 + z, t);
                nans[HD] = 1;
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::B_KV_FULL + stage));
        if (++stage == CH_STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      scale_slot = (scale_slot + 1) & 3;
    }
  }
}

// ------------------------------------------------------------------ MMA issue (1 thread)
template <int HD>
__device__ __forceinline__ void ch_issue_qk(uint32_t sbase, uint32_t tmem, int t, int kstage) {
  using L = ChLayout<HD>;
  constexpr uint32_t IDESC = idesc_f16_f32(CH_BM, CH_BN, 0, 0);
  const uint32_t qa = sbase + L::Q_OFF + t * L::TILE_BYTES;
  const uint32_t ka = sbase + L::KV_OFF + kstage * L::TILE_BYTES;
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) {
    const uint32_t off = (kk >> 2) * L::SUB_BYTES + (kk & 3) * 32;
    umma_ss(tmem + L::s_col(t), sdesc_sw128(qa + off, 16, 1024), sdesc_sw128(ka + off, 16, 1024), IDESC, kk > 0 ? 1u : 0u);
  }
}
template <int HD>
__device__ __forceinline__ void ch_issue_pv(uint32_t sbase, uint32_t tmem, int t, int vstage, bool accumulate) {
  using L = ChLayout<HD>;
  constexpr uint32_t IDESC = idesc_f16_f32(CH_BM, HD, 0, 1);
  const uint32_t va = sbase + L::KV_OFF + vstage * L::TILE_BYTES;
#pragma unroll
  for (int kk = 0; kk < CH_BN / 16; ++kk)
    umma_ts(tmem + L::o_col(t), tmem + L::s_col(t) + kk * 8, sdesc_sw128(va + kk * 2048, L::SUB_BYTES, 1024), IDESC,
            (accumulate || kk > 0) ? 1u : 0u);
}

template <int HD>
__device__ void ch_issue(ChWalk w, uint32_t sbase, uint32_t tmem, volatile int* abort_flag) {
  using L = ChLayout<HD>;
  const uint32_t bars = sbase + L::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * i; };
  int stage = 0;
  uint32_t phase = 0, q_phase = 0, p_phase[2] = {0, 0};
  auto advance = [&] {
    if (++stage == CH_STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  };
  bool ok = true;
  for (bool go = w.next(true); go && ok; go = w.next(false)) {
    if (!mbar_wait(bar(L::B_Q_FULL), q_phase, abort_flag)) break;
    q_phase ^= 1u;
    tc_fence_after();
    int vprev = 0, n = 0;
    for (int tile = w.t0; tile < w.t1; ++tile, ++n) {
      const int ks = stage;
      if (!mbar_wait(bar(L::B_KV_FULL + ks), phase, abort_flag)) { ok = false; break; }
      advance();
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (n > 0) {
          if (!mbar_wait(bar(L::B_P_READY + t), p_phase[t], abort_flag)) { ok = false; break; }
          p_phase[t] ^= 1u;
          tc_fence_after();
          ch_issue_pv<HD>(sbase, tmem, t, vprev, n > 1);
          if (t == 1) tc_commit(bar(L::B_KV_EMPTY + vprev));
        }
        ch_issue_qk<HD>(sbase, tmem, t, ks);
        tc_commit(bar(L::B_S_FULL + t));
      }
      if (!ok) break;
      tc_commit(bar(L::B_KV_EMPTY + ks));
      const int vs = stage;
      if (!mbar_wait(bar(L::B_KV_FULL + vs), phase, abort_flag)) { ok = false; break; }
      advance();
      tc_fence_after();
      vprev = vs;
    }
    if (!ok) break;
    tc_commit(bar(L::B_Q_EMPTY));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (!mbar_wait(bar(L::B_P_READY + t), p_phase[t], abort_flag)) { ok = false; break; }
      p_phase[t] ^= 1u;
      tc_fence_after();
      ch_issue_pv<HD>(sbase, tmem, t, vprev, n > 1);
      tc_commit(bar(L::B_O_FINAL + t));
    }
    if (!ok) break;
    tc_commit(bar(L::B_KV_EMPTY + vprev));
  }
  tc_commit(bar(L::B_DRAIN));
  drain_wait(bar(L::B_DRAIN), 0);
}

// ------------------------------------------------------------------ softmax (128 threads a tile)
// Scores to log2 units: row and key scale.  Never 0, which would turn a masked -inf into NaN (scores of
// such scales are 0 in any case).
__device__ __forceinline__ float ch_factor(float row_scale, float key_scale) {
  return fmaxf(row_scale * key_scale, 1.17549435e-38f);
}
// The same, but NaN for a key scale of NaN.
__device__ __forceinline__ float ch_factor_nan(float row_scale, float key_scale) {
  float f;
  asm("max.NaN.f32 %0, %1, 0f00800000;" : "=f"(f) : "f"(row_scale * key_scale));
  return f;
}

// This thread's query row of the piece that `w` stands on, as fp16 at the row's own power of two, into its
// place in shared memory; returns the factor from its scores to log2 units (before the key scale).
template <int HD>
__device__ __forceinline__ float ch_load_q(int t, const AttendParams& p, const ChWalk& w, uint8_t* smem, uint32_t full_bar) {
  using L = ChLayout<HD>;
  const int row = threadIdx.x & 127;
  const int at = w.i * CH_ROWS + t * CH_BM + row;
  uint4 v[HD / 8];
#pragma unroll
  for (int i = 0; i < HD / 8; ++i) v[i] = make_uint4(0, 0, 0, 0);
  if (at < w.n() * p.g) {
    const int tt = at / p.g;
    const uint4* q = reinterpret_cast<const uint4*>(p.q + w.b * p.qb + (static_cast<long long>(w.h) * p.g + at - tt * p.g) * p.qh + tt * p.qt);
#pragma unroll
    for (int i = 0; i < HD / 8; ++i) v[i] = q[i];
  }
  // magnitudes order like their bits; what is not finite does not count
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < HD / 8; ++i)
    for (uint32_t x : {v[i].x, v[i].y, v[i].z, v[i].w}) top = __vmaxu2(top, finite_bits(x));
  const float amax = __uint_as_float(max(top >> 16, top & 0xffffu) << 16);
  const int up = amax > 0.f ? min(max(14 - exponent_of(amax), -113), 126) : 0;   // amax -> [2^14, 2^15)
  const float f = two_to(up);
  auto half2_of = [&](uint32_t x) { return pack_half2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
  uint8_t* dst = smem + L::Q_OFF + t * L::TILE_BYTES + row * 128;
#pragma unroll
  for (int i = 0; i < HD / 8; ++i)
    *reinterpret_cast<uint4*>(dst + (i >> 3) * L::SUB_BYTES + (((i & 7) ^ (row & 7)) << 4)) =
        make_uint4(half2_of(v[i].x), half2_of(v[i].y), half2_of(v[i].z), half2_of(v[i].w));
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(full_bar);
  return p.scale_log2 * two_to(-up);
}

template <int HD>
__device__ void ch_softmax(int t, const AttendParams& p, ChWalk w, int per, uint8_t* smem, uint32_t sbase, uint32_t tmem,
                           volatile int* abort_flag) {
  using L = ChLayout<HD>;
  const uint32_t bars = sbase + L::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * i; };
  const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t tS = lane_base + L::s_col(t), tO = lane_base + L::o_col(t);
  const ChScales* scales = reinterpret_cast<const ChScales*>(smem + L::SCALE_OFF);
  uint32_t s_phase = 0, o_phase = 0, q_phase = 1;
  int scale_slot = 0, piece = 0;
  bool go = w.next(true);
  float row_scale = go ? ch_load_q<HD>(t, p, w, smem, bar(L::B_Q_FULL)) : 0.f;
  for (; go; piece = piece == 2 ? 0 : piece + 1) {
    const int row0 = w.i * CH_ROWS, rows = min(CH_ROWS, w.n() * p.g - row0);
    const int r = t * CH_BM + row;                 // within the item
    const bool row_ok = r < rows;
    const int lim = row_ok ? w.limit(row0 + r) : w.len();
    const int lim_first = w.limit(row0 + min(t * CH_BM, rows - 1));
    float m_ref = -INFINITY, top = -INFINITY, K = 0.f, l = 0.f, unit = two_to(-7);   // R, R + K, 2^(K - 7)
    int n = 0;
    for (int tile = w.t0; tile < w.t1; ++tile, ++n) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(L::B_S_FULL + t), s_phase, abort_flag))) return;
      s_phase ^= 1u;
      tc_fence_after();
      uint32_t s[CH_BN];
#pragma unroll
      for (int c = 0; c < CH_BN / 32; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
      tmem_ld_wait();
      const ChScales* sc = scales + scale_slot;
      scale_slot = (scale_slot + 1) & 3;
      const int k0 = tile * CH_BN;
      if (k0 + CH_BN > lim_first) {
        const int left = lim - k0;
#pragma unroll
        for (int c = 0; c < CH_BN; ++c)
          if (c >= left) s[c] = __float_as_uint(-INFINITY);
      }
      float m_tile = -INFINITY, y_tile = -INFINITY;   // largest score, and largest with its value scale 2^(e + 7)
#pragma unroll
      for (int g1 = 0; g1 < 8; ++g1) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int c = 16 * g1; c < 16 * g1 + 16; c += 4) {
          a = fmax3(a, __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
          b = fmax3(b, __uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        }
        const float4 lot = sc->lot[g1];
        const float m = fmaxf(a, b) * ch_factor_nan(row_scale, lot.x);
        m_tile = fmaxf(m_tile, m);
        y_tile = fmaxf(y_tile, m + lot.y);
      }
      const bool raise = m_tile > m_ref + AT_RAISE || y_tile - AT_P_LOG2 > top + AT_RAISE;
      float f = 1.f;                               // what O has to be multiplied by
      if (raise) {
        const float m_new = fmaxf(m_ref, m_tile), y_new = fmaxf(top, y_tile - AT_P_LOG2);
        K = fminf(fmaxf(floorf(y_new - m_new), E_MIN), E_MAX);
        f = ex2_approx(top - (m_new + K));         // nothing seen yet: 0
        l *= ex2_approx(m_ref - m_new);
        m_ref = m_new;
        top = m_new + K;
        unit = two_to(static_cast<int>(K) - 7);
      }
      if (n > 0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll 1
        for (int c = 0; c < HD / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(tO + 16 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st16(tO + 16 * c, o);
        }
        tmem_st_wait();
      }
      const float neg_ref = (m_ref == -INFINITY) ? 0.f : -m_ref;
#pragma unroll
      for (int hh = 0; hh < 4; ++hh) {             // 32 keys -> 16 packed columns
        uint32_t pk[16];
#pragma unroll
        for (int g1 = 0; g1 < 2; ++g1) {
          const float4 lot = sc->lot[2 * hh + g1];
          const float k1 = ch_factor(row_scale, lot.x);
          const float a1 = neg_ref + fmaxf(lot.y - K, lot.w);
          const float2 k2 = make_float2(k1, k1), a2 = make_float2(a1, a1);
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int at = 32 * hh + 16 * g1 + 2 * c;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[at]), __uint_as_float(s[at + 1])), k2, a2);
            float2 e;
            e.x = ex2_approx(x.x);
            e.y = ex2_approx(x.y);
            acc = __fadd2_rn(acc, e);
            pk[8 * g1 + c] = pack_half2(e.x, e.y);
          }
          l = fmaf(acc.x + acc.y, fminf(unit * lot.z, AT_L_MOST), l);
        }
        tmem_st16(tS + 16 * hh, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::B_P_READY + t));
    }
    // the next piece's queries, so that its products can start under this one's end
    ChWalk after = w;
    go = after.next(false);
    if (go) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(L::B_Q_EMPTY), q_phase ^ 1u, abort_flag))) return;
      q_phase ^= 1u;
      row_scale = ch_load_q<HD>(t, p, after, smem, bar(L::B_Q_FULL));
    }
    if (!__all_sync(0xffffffffu, mbar_wait(bar(L::B_O_FINAL + t), o_phase, abort_flag))) return;
    o_phase ^= 1u;
    tc_fence_after();
    // ---- epilogue
    const bool whole = w.t0 == 0 && w.t1 == w.nt;
    const int c0 = w.first / per, c1 = (w.first + w.nt - 1) / per;
    if (!whole && static_cast<int>(blockIdx.x) == c0 && threadIdx.x == 0) p.split[blockIdx.x] = make_int4(c1, c0, w.b, w.h * p.n_blocks + w.i);
    int* nans = reinterpret_cast<int*>(smem + L::NAN_OFF) + (piece * 8 + (threadIdx.x >> 5)) * (HD + 4);
    const bool any_nan = *reinterpret_cast<volatile int*>(nans + HD) != 0;
    const int gr = row0 + r, tt = gr / p.g, hq = w.h * p.g + gr - tt * p.g;
    const long long at = (static_cast<long long>(w.b) * p.c.heads * p.g + hq) * p.T + tt;
    // a part: [HD / 4][256 rows][4], so that a warp's rows make whole lines, then m and l [256 rows][2]
    float4* part = reinterpret_cast<float4*>(p.part) +
                   static_cast<long long>(2 * blockIdx.x + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * CH_ROWS * (HD / 4 + 1) + r;
    const float inv = l > 0.f ? 1.f / l : l;     // nothing seen: 0; NaN stays
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
      uint32_t o[16];
      tmem_ld16(tO + 16 * c, o);
      tmem_ld_wait();
      float y[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = l == 0.f ? 0.f : __uint_as_float(o[i]) * inv * unit;
      if (any_nan) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (nans[16 * c + i] < lim) y[i] = __uint_as_float(0x7fffffffu);
      }
      if (row_ok) {
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            part[(4 * c + i) * CH_ROWS] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        } else if (p.o_f32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.o) + at * HD + 16 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at * HD + 16 * c);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
        }
      }
    }
    if (row_ok) {
      if (whole)
        p.lse[at] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
      else
        *reinterpret_cast<float2*>(part + HD / 4 * CH_ROWS) = make_float2(m_ref, l);
    }
    if (any_nan) {                               // the same in the whole warp: clear for three pieces on
      __syncwarp();
      for (int i = lane; i < HD; i += 32) nans[i] = INT_MAX;
      if (lane == 0) nans[HD] = 0;
    }
    w = after;
  }
}

// ------------------------------------------------------------------ kernel
template <int HD>
__global__ void __launch_bounds__(CH_THREADS, 1) chunk_kernel(const AttendParams p) {
  using L = ChLayout<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  int* prefix = reinterpret_cast<int*>(smem + L::BATCH_OFF);
  int *s_slot = prefix + p.B + 1, *s_len = s_slot + p.B, *s_n = s_len + p.B;
  __shared__ int s_start[4];
  const Pool& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    const uint32_t bars = sbase + L::BAR_OFF;
    for (int i = 0; i < L::NUM_BARS; ++i) {
      const bool conv = i >= L::B_KV_FULL && i < L::B_KV_FULL + CH_STAGES;
      const bool p_ready = i >= L::B_P_READY && i < L::B_P_READY + 2;
      mbar_init(bars + 8u * i, i == L::B_Q_FULL ? 8 : conv ? CH_CONV_WARPS : p_ready ? CH_BM : 1);
    }
    *abort_flag = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    p.split[blockIdx.x] = make_int4(-1, 0, 0, 0);   // unless a piece of this block says otherwise
    fence_mbar_init();
  }
  if (warp == CH_WARP_MMA) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < 24 * (HD + 4); i += CH_THREADS)
    reinterpret_cast<int*>(smem + L::NAN_OFF)[i] = i % (HD + 4) < HD ? INT_MAX : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what ran before on the stream is complete
  // ---- the batch: lengths, and the places that each sequence takes on the line (a warp a sequence)
  for (int b = warp; b < p.B; b += CH_THREADS / 32) {
    const int slot = p.slots[b];
    int len = 0, n = 0;
    if (slot >= 0 && slot < c.slots) {
      len = c.lens[slot];
      n = p.n_new ? p.n_new[b] : p.T;
      if (n < 0 || n > p.T || len < 0 || len > c.max_pages * static_cast<long long>(c.page)) {
        if (blockIdx.x == 0 && lane == 0) record_pages();
        n = 0;
      }
    } else if (slot != -1 && blockIdx.x == 0 && lane == 0) {
      record_pages();
    }
    const int items = (n * p.g + CH_ROWS - 1) / CH_ROWS;
    int sum = 0;
    for (int i = lane; i < items; i += 32) sum += ChWalk::tiles(len, n, p.g, p.causal, i) + CH_START;
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) {
      s_slot[b] = slot;
      s_len[b] = len;
      s_n[b] = n;
      prefix[b] = sum;                             // per head, for now
    }
  }
  __syncthreads();
  if (warp == 0) {                                 // prefix sums over the batch, times the heads
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      const int w = b < p.B ? prefix[b] * c.heads : 0;
      int s = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
      }
      __syncwarp();
      if (b < p.B) prefix[b] = carry + s - w;
      carry += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) prefix[p.B] = carry;
  }
  __syncthreads();
  const int total = prefix[p.B];
  const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), CH_LEAST);
  const int line0 = static_cast<int>(min(static_cast<long long>(total), static_cast<long long>(blockIdx.x) * per));
  const int line1 = min(total, line0 + per);
  if (warp == 0 && line0 < line1) {                // the item that this block's stretch starts in
    const int b = find_row(prefix, p.B, line0);
    const int per_head = (prefix[b + 1] - prefix[b]) / c.heads;
    const int h = (line0 - prefix[b]) / per_head;
    const int rest = line0 - prefix[b] - h * per_head;
    const int items = (s_n[b] * p.g + CH_ROWS - 1) / CH_ROWS;
    int done = 0, at = 0;
    for (int i0 = 0;; i0 += 32) {
      const int w = i0 + lane < items ? ChWalk::tiles(s_len[b], s_n[b], p.g, p.causal, i0 + lane) + CH_START : 0;
      int s = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, i0 + lane < items && done + s > rest);
      if (behind || i0 + 32 >= items) {
        const int k = behind ? __ffs(behind) - 1 : 0;
        at = i0 + k;
        done += __shfl_sync(0xffffffffu, s - w, k);
        break;
      }
      done += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) {
      s_start[0] = b;
      s_start[1] = h;
      s_start[2] = at;
      s_start[3] = prefix[b] + h * per_head + done + CH_START;
    }
  }
  bool padding = false;
  if (p.fill_o || p.fill_lse)
    for (int b = threadIdx.x; b < p.B; b += CH_THREADS) padding |= s_n[b] < p.T;
  tc_fence_before();
  if (__syncthreads_or(padding)) fill_padding<HD>(p, s_n);
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;");   // the join can be set up, and wait
  const uint32_t tmem = *tmem_holder;
  ChWalk w;
  w.p = &p;
  w.batch = prefix;
  w.x = line0;
  w.line1 = line1;
  w.b = line0 < line1 ? s_start[0] : 0;
  w.h = line0 < line1 ? s_start[1] : 0;
  w.i = line0 < line1 ? s_start[2] : 0;
  w.first = line0 < line1 ? s_start[3] : 0;
  w.nt = w.t0 = w.t1 = 0;

  if (warp >= 8) {
    regs_lower<CH_REGS_OTHER>();
    if (warp == CH_WARP_MMA) {
      if (lane == 0) ch_issue<HD>(w, sbase, tmem, abort_flag);
      __syncwarp();
    } else if (warp == CH_WARP_FETCH) {
      ch_fetch<HD>(p, w, smem, sbase, abort_flag);
    } else {
      ch_convert<HD>(p, w, smem, sbase, abort_flag);
    }
  } else {
    regs_raise<CH_REGS_SOFTMAX>();
    ch_softmax<HD>(warp >> 2, p, w, per, smem, sbase, tmem, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == CH_WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts that chunk_kernel left: block (c, x, y) has rows 32 y .. of the segment that starts in its
// block c, a row a lane, column group CHJ_WARPS x + warp a warp, all reads whole lines.
constexpr int CHJ_WARPS = 8;

template <int HD>
__global__ void __launch_bounds__(CHJ_WARPS * 32) chunk_join_kernel(const AttendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the parts are complete
  asm volatile("griddepcontrol.launch_dependents;");
  const int4 d = p.split[blockIdx.x];
  if (d.x < 0) return;
  const int c0 = d.y, n = d.x - c0 + 1, b = d.z, h = d.w / p.n_blocks, row0 = (d.w - h * p.n_blocks) * CH_ROWS;
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), group = blockIdx.z * CHJ_WARPS + (threadIdx.x >> 5);
  if (r >= min(CH_ROWS, (p.n_new ? p.n_new[b] : p.T) * p.g - row0)) return;
  constexpr long long PART = static_cast<long long>(CH_ROWS) * (HD / 4 + 1);
  const float4* parts = reinterpret_cast<const float4*>(p.part) + r;
  // part of block c0: its second place; of a block behind it: the first
  auto at = [&](int k) { return parts + (k ? 2ll * (c0 + k) : 2ll * c0 + 1) * PART; };
  float m = -INFINITY, z = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int LOT = 8;                               // parts read together
  for (int k0 = 0; k0 < n; k0 += LOT) {
    float2 ml[LOT];
    float4 y[LOT];
#pragma unroll
    for (int k = 0; k < LOT; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (k0 + k < n) {
        ml[k] = *reinterpret_cast<const float2*>(at(k0 + k) + HD / 4 * CH_ROWS);
        y[k] = at(k0 + k)[group * CH_ROWS];
      }
    }
    join_parts<false>(ml, y, m, z, a);
  }
  store_row<HD>(p, b, h, row0 + r, 4 * group, m, z, a);
}

}  // namespace cache
}  // namespace ra
