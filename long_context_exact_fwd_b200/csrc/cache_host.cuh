// Host side of the 8-bit key/value cache: argument checks, workspaces and launches.  Included once,
// at the end of ring_attn.cu (it uses that file's device info, status and alignment helpers).
#pragma once
#include "cache.cuh"
#include "cache_attn.cuh"
#include "cache_chunk.cuh"
#include "cache_io.cuh"
#include "cache_pages.cuh"

namespace {

namespace rc = ra::cache;

// Shared memory of the attention kernels set on this device: [Dh 128, Dh 64][8-row column blocks - 1, then chunks].
std::atomic<bool> g_attend_set[MAX_DEVICES][2][4];

// Checks the description of a cache and fills `p` with all layers' view; layer >= 0 picks one.
int cache_pool(const ra_cache* c, int layer, rc::Pool* p) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !c->lens || !c->refs) return RA_ERR_ARG;
  if (c->layers <= 0 || c->pages <= 0 || c->heads <= 0 || c->slots <= 0 || c->max_pages <= 0) return RA_ERR_ARG;
  if (layer >= c->layers) return RA_ERR_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return RA_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return RA_ERR_SHAPE;
  // positions fit in int (with a tile to spare), page numbers and per-layer head indexes too
  if (static_cast<long long>(c->max_pages) * c->page > INT_MAX - 1024) return RA_ERR_SHAPE;
  // nor may a batch's pages, at most every entry of the table and a copy each, pass it: plans add them up
  if (static_cast<long long>(c->slots) * c->max_pages > INT_MAX - 2 * rc::MAX_BATCH) return RA_ERR_SHAPE;
  if (c->pages > (1 << 28) || c->heads > 32767 || c->layers > (1 << 20)) return RA_ERR_SHAPE;
  if (static_cast<double>(c->layers) * c->pages * c->heads * c->page * c->head_dim > 9.0e18 / 4) return RA_ERR_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v)) return RA_ERR_ALIGN;
  for (const void* q : {static_cast<const void*>(c->k_scale), static_cast<const void*>(c->v_scale),
                        static_cast<const void*>(c->table), static_cast<const void*>(c->lens),
                        static_cast<const void*>(c->refs)})
    if (reinterpret_cast<uintptr_t>(q) % 4) return RA_ERR_ALIGN;
  const long long rows = layer > 0 ? static_cast<long long>(layer) * c->pages * c->heads : 0;
  const long long codes = rows * c->page * c->head_dim;
  *p = {static_cast<uint8_t*>(c->k) + codes, static_cast<uint8_t*>(c->v) + codes, c->k_scale + rows, c->v_scale + rows,
        c->table, c->lens, c->refs, c->layers, c->pages, c->heads, c->page, c->head_dim, c->slots, c->max_pages};
  return RA_OK;
}

int cache_batch(const int* slots, int B) {
  if (!slots || B <= 0) return RA_ERR_ARG;
  if (B > rc::MAX_BATCH) return RA_ERR_SHAPE;
  return reinterpret_cast<uintptr_t>(slots) % 4 ? RA_ERR_ALIGN : RA_OK;
}

// Rows of a [B][heads][T][Dh] bf16 tensor that kernels read 16 bytes at a time.
int cache_rows(const void* x, const long long* st, int B, int H, int T) {
  if (!x || !st) return RA_ERR_ARG;
  const int n[3] = {B, H, T};
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (st[i] < 0 || st[i] > (1ll << 59) / n[i]) return RA_ERR_SHAPE;
    if (st[i] % 8) return RA_ERR_ALIGN;
  }
  return aligned16(x) ? RA_OK : RA_ERR_ALIGN;
}

// Whether `a_bytes` from a and `b_bytes` from b have a byte in common.
bool overlap(const void* a, unsigned long long a_bytes, const void* b, unsigned long long b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

size_t pages_workspace(long long words) { return align256(sizeof(rc::Plan)) + align256(static_cast<size_t>(words) * 4); }

int pages_check_ws(const void* workspace, size_t have, size_t need) {
  return !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || have < need ? RA_ERR_WORKSPACE : RA_OK;
}

int copy_grid(const rc::Pool& c, long long pairs, int sm_count) {
  const long long chunks = (static_cast<long long>(c.heads) * c.page * c.Dh + rc::COPY_BYTES - 1) / rc::COPY_BYTES;
  const long long units = pairs * c.layers * 2 * chunks;
  const long long most = 8ll * sm_count;   // resident at 256 threads
  return static_cast<int>(units < 1 ? 1 : (units < most ? units : most));
}

// Which kernel a call's rows per kv head (T * g) take: 0 is chunk_kernel; otherwise attend_kernel with
// blocks of 8 * nt rows, as few blocks as 24 rows allow and the narrowest that do.  Measured, attend_kernel
// and chunk_kernel, 4 query heads on each of 8 of 128: 16 contexts up to 4K, 48 rows 66 and 68 us, 64 rows 90
// and 68, 128 rows 153 and 74; one context of 32K, 48 rows 46 and 55, 64 rows 60 and 55, 128 rows 101 and 57; one of
// 4K, where neither is busy, 64 rows 23 and 27 (the host does not know the lengths).
constexpr int CHUNK_ROWS = 64;
// Calls of so few segments join them with a block per row and 16 warps (4 warps a row otherwise).  Measured, 16
// warps and 4: one segment of 128K tokens (444 parts) 17.7 and 27.4 us, eight of them 49.9 and 51.5, eight of 8K
// 12.4 and 12.1, 16 of 777 11.2 and 9.9.
constexpr int FEW_SEGMENTS = 8;
constexpr int AT_MAX_NT = 3;
int attend_nt(long long rows) {
  if (rows >= CHUNK_ROWS) return 0;
  const long long blocks = (rows + 8 * AT_MAX_NT - 1) / (8 * AT_MAX_NT);
  return static_cast<int>((rows + 8 * blocks - 1) / (8 * blocks));
}

// A launch that may be set up while the kernel before it on the stream still runs; every kernel of the cache
// waits for that one's end (behind_last) before it touches memory.
template <typename... P, typename... A>
int launch_behind(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) return cuda_fail(static_cast<int>(e), "cudaLaunchKernelEx(cache)");
  return launch_status();
}

// Shared memory of a kernel, set once per device.
template <typename K>
int attend_smem(std::atomic<bool>& set, K kernel, int most) {
  if (set) return RA_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return cuda_fail(static_cast<int>(e), "cudaFuncSetAttribute(cache attention smem)");
  set = true;
  return RA_OK;
}

template <int HD, int NT>
int attend_launch(const rc::AttendParams& p, DevInfo* di, cudaStream_t stream) {
  int st = attend_smem(g_attend_set[di - g_dev][HD == 128 ? 0 : 1][NT - 1], rc::attend_kernel<HD, NT>,
                       rc::AttLayout<HD, NT>::bytes(rc::MAX_BATCH));
  if (st != RA_OK) return st;
  const int grid = rc::at_per_sm(HD, NT) * (di->sm_count < rc::AT_MAX_SMS ? di->sm_count : rc::AT_MAX_SMS);
  st = launch_behind(rc::attend_kernel<HD, NT>, dim3(grid), rc::AT_THREADS, rc::AttLayout<HD, NT>::bytes(p.B), stream, p);
  if (st != RA_OK) return st;
  if (p.by_segment)   // few segments, many parts each: a block per row, 16 warps
    return launch_behind(rc::join_kernel<HD, 8 * NT, 1, 16>, dim3(p.B * p.c.heads * p.n_blocks, 8 * NT), 512, 0, stream, p);
  return launch_behind(rc::join_kernel<HD, 8 * NT, 2, 4>, dim3(grid, 4 * NT), 256, 0, stream, p);
}

template <int HD>
int chunk_launch(const rc::AttendParams& p, DevInfo* di, cudaStream_t stream) {
  int st = attend_smem(g_attend_set[di - g_dev][HD == 128 ? 0 : 1][AT_MAX_NT], rc::chunk_kernel<HD>,
                       rc::ChLayout<HD>::bytes(rc::MAX_BATCH));
  if (st != RA_OK) return st;
  const int grid = di->sm_count < rc::CH_MAX_CTAS ? di->sm_count : rc::CH_MAX_CTAS;
  st = launch_behind(rc::chunk_kernel<HD>, dim3(grid), rc::CH_THREADS, rc::ChLayout<HD>::bytes(p.B), stream, p);
  if (st != RA_OK) return st;
  return launch_behind(rc::chunk_join_kernel<HD>, dim3(grid, rc::CH_ROWS / 32, HD / 4 / rc::CHJ_WARPS), rc::CHJ_WARPS * 32, 0,
                       stream, p);
}

template <int HD>
int attend_dispatch(int nt, const rc::AttendParams& p, DevInfo* di, cudaStream_t stream) {
  if (nt == 0) return chunk_launch<HD>(p, di, stream);
  if (nt == 1) return attend_launch<HD, 1>(p, di, stream);
  if (nt == 2) return attend_launch<HD, 2>(p, di, stream);
  return attend_launch<HD, 3>(p, di, stream);
}

size_t attend_part_bytes(int nt, int Dh) {
  const size_t parts = nt ? 2ull * rc::at_per_sm(Dh, nt) * rc::AT_MAX_SMS * 8 * nt : 2ull * rc::CH_MAX_CTAS * rc::CH_ROWS;
  return align256(parts * (Dh + 4) * sizeof(float));
}

}  // namespace

extern "C" {

int ring_attn_cache_append(const ra_cache* cache, int layer, const int* slots, const int* n_new, int B, int T,
                           const void* k, const long long* k_strides, const void* v, const long long* v_strides,
                           ra_stream stream) {
  rc::AppendParams p{};
  if (layer < 0 || T <= 0) return RA_ERR_ARG;
  int st = cache_pool(cache, layer, &p.c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(slots, B)) != RA_OK) return st;
  if ((st = cache_rows(k, k_strides, B, p.c.heads, T)) != RA_OK) return st;
  if ((st = cache_rows(v, v_strides, B, p.c.heads, T)) != RA_OK) return st;
  if (reinterpret_cast<uintptr_t>(n_new) % 4) return RA_ERR_ALIGN;
  if (T > INT_MAX - 1024) return RA_ERR_SHAPE;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.kb = k_strides[0], p.kh = k_strides[1], p.kt = k_strides[2];
  p.vb = v_strides[0], p.vh = v_strides[1], p.vt = v_strides[2];
  p.slots = slots;
  p.n_new = n_new;
  p.T = T;
  const long long touched = (T + static_cast<long long>(p.c.page) - 2) / p.c.page + 1;   // pages T tokens can lie in
  const long long most = touched < p.c.max_pages ? touched : p.c.max_pages;
  const dim3 grid(static_cast<unsigned>(most), p.c.heads, 2 * B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int units = p.c.page * p.c.Dh / rc::UNIT;
  void (*kernel)(rc::AppendParams) = units <= rc::AP_THREADS       ? rc::append_kernel<1>
                                     : units <= 2 * rc::AP_THREADS ? rc::append_kernel<2>
                                     : units <= 4 * rc::AP_THREADS ? rc::append_kernel<4>
                                     : units <= 8 * rc::AP_THREADS ? rc::append_kernel<8>
                                                                   : rc::append_kernel<16>;
  return launch_behind(kernel, grid, rc::AP_THREADS, 0, s, p);
}

int ring_attn_cache_read(const ra_cache* cache, int layer, const int* slots, const int* start, int B, int length,
                         void* k, void* v, ra_stream stream) {
  return ring_attn_cache_read_ex(cache, layer, slots, start, B, length, k, v, 0, 0, stream);
}

int ring_attn_cache_read_ex(const ra_cache* cache, int layer, const int* slots, const int* start, int B, int length,
                            void* k, void* v, int fill_k, int fill_v, ra_stream stream) {
  rc::ReadParams p{};
  if (layer < 0 || length <= 0 || !k || !v || k == v) return RA_ERR_ARG;
  int st = cache_pool(cache, layer, &p.c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(slots, B)) != RA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || reinterpret_cast<uintptr_t>(start) % 4) return RA_ERR_ALIGN;
  const unsigned long long bytes = 2ull * B * p.c.heads * length * p.c.Dh;
  if (overlap(k, bytes, v, bytes)) return RA_ERR_ARG;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  p.slots = slots;
  p.start = start;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.length = length;
  p.fill_k = fill_k != 0;
  p.fill_v = fill_v != 0;
  const int per_block = rc::READ_UNITS * rc::IO_THREADS * rc::UNIT / p.c.Dh;   // tokens
  const dim3 grid((length + static_cast<long long>(per_block) - 1) / per_block, p.c.heads, 2 * B);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return launch_behind(p.c.Dh == 128 ? rc::read_kernel<128> : rc::read_kernel<64>, grid, rc::IO_THREADS, 0, s, p);
}

size_t ring_attn_cache_attend_workspace_size(int T, int Hq, int Hkv, int Dh) {
  if (T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (Dh != 64 && Dh != 128)) return 0;
  const int nt = attend_nt(static_cast<long long>(T) * (Hq / Hkv));
  return attend_part_bytes(nt, Dh) + align256(4 * rc::AT_MAX_SMS * sizeof(int4))   /* blocks: at_per_sm per SM, at most 4 */;
}

int ring_attn_cache_attend(const ra_cache* cache, int layer, const int* slots, const int* n_new, int B, int T, int Hq,
                           const void* q, const long long* q_strides, float scale, int causal, void* o,
                           ra_dtype o_dtype, float* lse, void* workspace, size_t workspace_bytes, ra_stream stream) {
  return ring_attn_cache_attend_ex(cache, layer, slots, n_new, B, T, Hq, q, q_strides, scale, causal, o, o_dtype, lse, 0, 0,
                                   workspace, workspace_bytes, stream);
}

int ring_attn_cache_attend_ex(const ra_cache* cache, int layer, const int* slots, const int* n_new, int B, int T, int Hq,
                              const void* q, const long long* q_strides, float scale, int causal, void* o,
                              ra_dtype o_dtype, float* lse, int fill_o, int fill_lse, void* workspace,
                              size_t workspace_bytes, ra_stream stream) {
  rc::AttendParams p{};
  if (layer < 0 || T <= 0 || Hq <= 0 || !o || !lse) return RA_ERR_ARG;
  if (o_dtype != RA_BF16 && o_dtype != RA_F32) return RA_ERR_ARG;
  int st = cache_pool(cache, layer, &p.c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(slots, B)) != RA_OK) return st;
  if (Hq % p.c.heads) return RA_ERR_SHAPE;
  if ((st = cache_rows(q, q_strides, B, Hq, T)) != RA_OK) return st;
  if (!aligned16(o) || reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(n_new) % 4) return RA_ERR_ALIGN;
  // rows are written while others' queries are still read: the outputs may not lie over the queries, nor each other
  const auto reach = [&](int i, int n) { return n > 1 ? q_strides[i] * (n - 1) : 0; };
  const unsigned long long q_bytes = 2ull * (reach(0, B) + reach(1, Hq) + reach(2, T) + p.c.Dh);
  const unsigned long long lse_bytes = 4ull * B * Hq * T, o_bytes = lse_bytes / 4 * p.c.Dh * (o_dtype == RA_F32 ? 4 : 2);
  if (overlap(q, q_bytes, o, o_bytes) || overlap(q, q_bytes, lse, lse_bytes) || overlap(o, o_bytes, lse, lse_bytes))
    return RA_ERR_ARG;
  p.g = Hq / p.c.heads;
  const long long rows = static_cast<long long>(T) * p.g;
  if (rows > INT_MAX / 2) return RA_ERR_SHAPE;
  const int nt = attend_nt(rows);
  // rows per block, and the line of places, which is numbered in int
  const int block = nt ? 8 * nt : rc::CH_ROWS, tile = nt ? rc::AT_TILE : rc::CH_BN, start = nt ? rc::AT_START : rc::CH_START;
  p.n_blocks = static_cast<int>((rows + block - 1) / block);
  // up to so many segments, each is likely split: one entry per segment, and the wide join
  p.by_segment = static_cast<long long>(B) * p.c.heads * p.n_blocks <= FEW_SEGMENTS;
  const double places = std::ceil(static_cast<double>(p.c.max_pages) * p.c.page / tile) + start;
  if (places * p.c.heads * p.n_blocks * B > INT_MAX / 2) return RA_ERR_SHAPE;
  if ((st = pages_check_ws(workspace, workspace_bytes, ring_attn_cache_attend_workspace_size(T, Hq, p.c.heads, p.c.Dh))) != RA_OK)
    return st;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.qb = q_strides[0], p.qh = q_strides[1], p.qt = q_strides[2];
  p.slots = slots;
  p.n_new = n_new;
  p.o = o;
  p.lse = lse;
  p.fill_o = fill_o != 0;
  p.fill_lse = fill_lse != 0;
  p.part = static_cast<float*>(workspace);
  p.split = reinterpret_cast<int4*>(static_cast<char*>(workspace) + attend_part_bytes(nt, p.c.Dh));
  p.B = B;
  p.T = T;
  p.page_shift = p.c.page == 16 ? 4 : p.c.page == 32 ? 5 : p.c.page == 64 ? 6 : 7;
  p.causal = causal != 0;
  p.o_f32 = o_dtype == RA_F32;
  const float sc = (scale > 0.f && std::isfinite(scale)) ? scale : 1.0f / std::sqrt(static_cast<float>(p.c.Dh));
  p.scale_log2 = sc * 1.4426950408889634f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p.c.Dh == 128 ? attend_dispatch<128>(nt, p, di, s) : attend_dispatch<64>(nt, p, di, s);
}

size_t ring_attn_cache_pages_workspace_size(int B, int pages) {
  if (B < 0 || pages <= 0) return 0;
  return pages_workspace(3ll * pages + 2ll * B + 1);
}

int ring_attn_cache_reserve(const ra_cache* cache, const int* slots, const int* n_new, int B, void* workspace,
                            size_t workspace_bytes, ra_stream stream) {
  return ring_attn_cache_reserve_ex(cache, slots, n_new, B, nullptr, workspace, workspace_bytes, stream);
}

int ring_attn_cache_reserve_ex(const ra_cache* cache, const int* slots, const int* n_new, int B, int* granted,
                               void* workspace, size_t workspace_bytes, ra_stream stream) {
  rc::Pool c;
  int st = cache_pool(cache, -1, &c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(slots, B)) != RA_OK) return st;
  if (!n_new) return RA_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(n_new) % 4 || reinterpret_cast<uintptr_t>(granted) % 4) return RA_ERR_ALIGN;
  // written while slots and other counts may still be read
  if (granted && (overlap(granted, 4ull * B, slots, 4ull * B) ||
                  (granted != n_new && overlap(granted, 4ull * B, n_new, 4ull * B))))
    return RA_ERR_ARG;
  if ((st = pages_check_ws(workspace, workspace_bytes, ring_attn_cache_pages_workspace_size(B, c.pages))) != RA_OK) return st;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc::Plan* plan = static_cast<rc::Plan*>(workspace);
  int* pairs = reinterpret_cast<int*>(static_cast<char*>(workspace) + align256(sizeof(rc::Plan)));
  int* free_list = pairs + 2 * B;
  st = launch_behind(rc::reserve_plan_kernel, dim3(1), rc::PLAN_THREADS, 0, s, c, slots, n_new, B, granted, plan, pairs,
                     free_list);
  if (st != RA_OK) return st;
  return launch_behind(rc::copy_pages_kernel, dim3(copy_grid(c, B, di->sm_count)), rc::COPY_THREADS, 0, s, c, plan, pairs,
                       pairs + 1, 2, nullptr);
}

int ring_attn_cache_fork(const ra_cache* cache, const int* src, const int* dst, int B, void* workspace,
                         size_t workspace_bytes, ra_stream stream) {
  rc::Pool c;
  int st = cache_pool(cache, -1, &c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(src, B)) != RA_OK || (st = cache_batch(dst, B)) != RA_OK) return st;
  if ((st = pages_check_ws(workspace, workspace_bytes, ring_attn_cache_pages_workspace_size(B, c.pages))) != RA_OK) return st;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc::Plan* plan = static_cast<rc::Plan*>(workspace);
  int* first = reinterpret_cast<int*>(static_cast<char*>(workspace) + align256(sizeof(rc::Plan)));
  st = launch_behind(rc::fork_plan_kernel, dim3(1), rc::PLAN_THREADS, 0, s, c, src, dst, B, plan, first);
  if (st != RA_OK) return st;
  const long long items = static_cast<long long>(B) * c.max_pages;
  const long long blocks = (items + rc::COPY_THREADS - 1) / rc::COPY_THREADS;
  const int grid = static_cast<int>(blocks < 2ll * di->sm_count ? blocks : 2ll * di->sm_count);
  return launch_behind(rc::fork_apply_kernel, dim3(grid), rc::COPY_THREADS, 0, s, c, src, dst, plan, first);
}

int ring_attn_cache_trim(const ra_cache* cache, const int* slots, const int* keep, int B, ra_stream stream) {
  rc::Pool c;
  int st = cache_pool(cache, -1, &c);
  if (st != RA_OK) return st;
  if ((st = cache_batch(slots, B)) != RA_OK) return st;
  if (reinterpret_cast<uintptr_t>(keep) % 4) return RA_ERR_ALIGN;
  if (!dev_info(&st)) return st;
  return launch_behind(rc::trim_kernel, dim3(B), rc::COPY_THREADS, 0, static_cast<cudaStream_t>(stream), c, slots, keep, B);
}

int ring_attn_cache_compact(const ra_cache* cache, void* workspace, size_t workspace_bytes, ra_stream stream) {
  rc::Pool c;
  int st = cache_pool(cache, -1, &c);
  if (st != RA_OK) return st;
  if ((st = pages_check_ws(workspace, workspace_bytes, ring_attn_cache_pages_workspace_size(0, c.pages))) != RA_OK) return st;
  DevInfo* di = dev_info(&st);
  if (!di) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  rc::Plan* plan = static_cast<rc::Plan*>(workspace);
  int* holes = reinterpret_cast<int*>(static_cast<char*>(workspace) + align256(sizeof(rc::Plan)));
  int *movers = holes + c.pages, *moved_to = movers + c.pages;
  st = launch_behind(rc::compact_plan_kernel, dim3(1), rc::PLAN_THREADS, 0, s, c, plan, holes, movers, moved_to);
  if (st != RA_OK) return st;
  const int grid = copy_grid(c, c.pages / 2 + 1, di->sm_count);
  return launch_behind(rc::copy_pages_kernel, dim3(grid), rc::COPY_THREADS, 0, s, c, plan, movers, holes, 1, moved_to);
}

}  // extern "C"
