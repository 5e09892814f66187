// libmpzch: C entry points of the history cache (include/mpzch.h, "History
// cache").
#include "mpzch.h"
#include "mpzch_internal.h"
#include "mpzch_kv_rows.cuh"
#include "mpzch_kv_tiles.cuh"
#include "mpzch_launch.cuh"

#include <cmath>

using namespace mpzch_kv;
using namespace mpzch_internal;

namespace {

constexpr int64_t kMaxInt = 0x7FFFFFFFll;
constexpr float kLog2E = 1.4426950408889634f;

int log2_of(int x) {
  int k = 0;
  while ((1 << k) < x) ++k;
  return k;
}

bool block_size_ok(int32_t s) { return s == 16 || s == 32 || s == 64 || s == 128; }
bool dim_ok(int32_t d) { return d == 32 || d == 64 || d == 128; }
int type_bytes(int32_t t) {
  return t == MPZCH_F32 ? 4 : t == MPZCH_F16 || t == MPZCH_BF16 ? 2 : 0;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Rows of heads: every head of every row starts on a 16-byte boundary.
bool rows_ok(const void* p, int64_t sn, int64_t sh, int bytes) {
  return aligned16(p) && sn >= 0 && sh >= 0 && (sn * bytes) % 16 == 0 && (sh * bytes) % 16 == 0 &&
         sn < (1ll << 40) && sh < (1ll << 40);
}

// Whether any two of n x h heads of `dim` elements, sn and sh elements apart, share one.  Where
// one stride passes all that lies in the other (every ordinary view) that is seen at once;
// else, for each distance in heads, the two nearest distances in rows are looked at.
bool heads_overlap(int64_t n, int64_t sn, int64_t h, int64_t sh, int64_t dim) {
  if ((n > 1 && sn < dim) || (h > 1 && sh < dim)) return true;
  if (n <= 1 || h <= 1 || sn >= (h - 1) * sh + dim || sh >= (__int128)(n - 1) * sn + dim)
    return false;
  for (int64_t j = 1; j < h; ++j) {
    const int64_t i = j * sh / sn, off = j * sh - i * sn;  // 0 <= off < sn
    if ((i < n && off < dim) || (i + 1 < n && sn - off < dim)) return true;
  }
  return false;
}

template <typename T, int D, int W>
int launch_append(const AppendArgs& a, cudaStream_t st) {
  const void* kern = reinterpret_cast<const void*>(k_kv_append<T, D, W>);
  // blocks for one head and cache: for all rows, or for what is resident
  const int64_t groups = (a.n + a.rows_per_warp - 1) / a.rows_per_warp;
  int64_t y = (groups + 8 / W - 1) / (8 / W);
  const int64_t most = (int64_t)sm_count() * resident_blocks(kern, 256, 0) / (2 * a.H);
  if (y > most) y = most < 1 ? 1 : most;
  return launch(k_kv_append<T, D, W>, dim3(2 * a.H, (unsigned)y), 256, st, true, a);
}

template <typename T, int D>
int launch_append_warps(const AppendArgs& a, cudaStream_t st) {
  const int w = append_warps(D, 1 << a.bs_log);
  if constexpr (append_warps(D, 128) >= 8)
    if (w == 8) return launch_append<T, D, 8>(a, st);
  if constexpr (append_warps(D, 128) >= 4)
    if (w == 4) return launch_append<T, D, 4>(a, st);
  return w == 2 ? launch_append<T, D, 2>(a, st) : launch_append<T, D, 1>(a, st);
}

template <typename T>
int launch_append_dim(const AppendArgs& a, int dim, cudaStream_t st) {
  return dim == 32 ? launch_append_warps<T, 32>(a, st)
                   : dim == 64 ? launch_append_warps<T, 64>(a, st)
                               : launch_append_warps<T, 128>(a, st);
}

// (the join's table of weights holds the parts of all workers)
int row_workers() {
  const int n = sm_count() * kRowBlocksPerSm * kRowWarps;
  return n < kMostParts ? n : kMostParts;
}

int64_t head_bytes() {
  return (row_workers() * (int64_t)sizeof(PartHead) + 255) / 256 * 256;
}

int64_t part_bytes(int dim) {
  const int64_t rows = row_workers() * 2ll * kMaxRows, tiles = sm_count() * 2ll * kTileRows;
  return head_bytes() + (rows > tiles ? rows : tiles) * (dim + 2) * (int64_t)sizeof(float);
}

template <int D, typename T>
int launch_tiles(const AttendArgs& a, cudaStream_t st) {
  constexpr int kBytes = TileSmem<D>::kBytes;
  const unsigned grid = (unsigned)sm_count();
  int rc = launch_smem(k_kv_tiles<D, T>, grid, kTileThreads, kBytes, st, true, a);
  if (!rc)
    rc = launch(k_kv_join<D, T, kTileRows>, dim3(grid, kTileRows / kJoinWarps), 32 * kJoinWarps, st,
                true, a, (int)grid);
  return rc;
}

// What the table has room for decides, since the host knows no length: where that is
// kWholeKeys at most and the items (request, kv head) are few, each goes whole to a warp: its
// 32 steps take about as long as the launch that would join the parts of cut ones (4
// requests x 8 heads of up to 300 keys, dim 64, on the device: one launch 11.5 us, cut and
// joined 8.5 + 5.1 us; and a caller issues one launch fewer, 16.6 against 18.5 us a call).
// Many items balance better cut (128 x 8 of up to 500 keys 17 us, whole 22; 366 x 8 of up to
// 271 keys 26 : 31), unless they are a step or two long (1,749 x 8 of up to 3 keys, 8 query
// heads each: 33 us, whole 30).
constexpr int64_t kTinyKeys = 128, kWholeItems = 256;
constexpr int64_t kWholeKeys = 512;

template <int D, typename T, int R, int NQ, int NP>
int launch_rows(const AttendArgs& a, cudaStream_t st) {
  const void* kern = reinterpret_cast<const void*>(k_kv_rows<D, T, R, NQ, NP>);
  int rc = allow_dynamic_smem(kern, row_smem(D));
  if (rc) return rc;
  int per_sm = resident_blocks(kern, 32 * kRowWarps, row_smem(D));
  if (per_sm > kRowBlocksPerSm) per_sm = kRowBlocksPerSm;
  unsigned grid = (unsigned)(sm_count() * per_sm);
  if (grid > (unsigned)row_workers() / kRowWarps) grid = row_workers() / kRowWarps;
  rc = launch_smem(k_kv_rows<D, T, R, NQ, NP>, grid, 32 * kRowWarps, row_smem(D), st, true, a);
  if (a.unit_keys != kUnitKeys) return rc;  // no item is cut
  // Items cut into many parts want a block for each row, and there are only a few of
  // them; where there are many items, most blocks have nothing to join or a few parts,
  // and a warp for every second row of their items is enough (64 x 1..7 drafts, 8 query
  // heads to a kv head: 21.4 us with R / 4 blocks across, 27.2 with R).
  const int64_t rows = (int64_t)a.max_new * a.G;
  const int y = (int64_t)a.B * a.H > 64 ? R / 4 : rows < 1 ? 1 : rows < R ? (int)rows : R;
  if (!rc)
    rc = launch(k_kv_join<D, T, R>, dim3((grid * kRowWarps + join_heads<R>() - 1) / join_heads<R>(), y),
                32 * kJoinWarps, st, true, a, (int)(grid * kRowWarps));
  return rc;
}

// Tiles of 8 rows where no request has more, else of 16; 16-bit types with more rows go
// to the tile kernel.  A half tile of it costs the same for 20 rows as for 128, and a
// block takes one item at a time, so many requests with up to 32 (dim 128) or 64 (dim 64)
// rows stay here.  Row kernel against tile kernel, us on the device: 64 requests x 8 kv
// heads x 20 rows, dim 128, up to 512 keys 35 : 50; 128 x 2 x 32 rows, dim 128, 1,000 to 4,000
// keys 89 : 112; 64 x 2 x 56 rows, dim 64, window 1,024 21 : 29, all of up to 8,192 keys
// 36 : 38; but 32 x 2 x 32 rows, dim 128 42 : 39; 16 x 8 x 32 rows, up to 512 keys 39 : 25;
// 8 x 2 x 20 rows, up to 1,000 keys 24 : 17.
template <int D, typename T, int NQ, int NP>
int launch_rows(const AttendArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.G;
  if constexpr (D >= 64 && sizeof(T) == 2) {
    if (rows > 16 && (a.B < 64 || rows * D > 4096)) return launch_tiles<D, T>(a, st);
  }
  return rows <= 8 ? launch_rows<D, T, 8, NQ, NP>(a, st) : launch_rows<D, T, 16, NQ, NP>(a, st);
}

// NQ, NP: fp16 parts of the queries and of the weights.  16-bit queries fit one part (rows
// are scaled by a power of two).  Weights in one part, 11 bits, are what bf16 results get:
// single tokens of 256 requests are then 1.670e-3 from 64 bits (relative, over all
// outputs) where weights in 32 bits give 1.656e-3, nearly all of both the rounding of the
// result; fp16 results would be 1.4 times as far as that rounding, so they take two.
template <typename T, int NQ, int NP>
int launch_rows_dim(const AttendArgs& a, int dim, cudaStream_t st) {
  return dim == 32 ? launch_rows<32, T, NQ, NP>(a, st)
                   : dim == 64 ? launch_rows<64, T, NQ, NP>(a, st) : launch_rows<128, T, NQ, NP>(a, st);
}

}  // namespace

extern "C" {

int mpzch_kv_tables(const int32_t* cached_len, const int32_t* new_len, int32_t n_requests,
                    int32_t block_size, const int32_t* free_blocks, int64_t n_free_blocks,
                    const int64_t* free_count, int32_t* block_table, int32_t max_blocks,
                    int32_t* cu_new, int32_t* seq_len, int64_t* slots, int64_t n_slots,
                    int64_t* free_count_out, int32_t* dev_status, void* stream) {
  if (n_requests < 0 || n_requests > MPZCH_KV_MAX_REQUESTS || !block_size_ok(block_size) ||
      n_free_blocks < 0 || n_free_blocks >= kMaxInt || max_blocks < 0 ||
      (int64_t)max_blocks * block_size > kMaxInt - 1024 || n_slots < 0 || n_slots >= kMaxInt)
    return MPZCH_EINVAL;
  if (!free_count || !free_count_out || free_count == free_count_out || !cu_new ||
      (n_free_blocks > 0 && !free_blocks) || (n_slots > 0 && !slots))
    return MPZCH_EINVAL;
  if (n_requests > 0 && (!cached_len || !new_len || !seq_len || (max_blocks > 0 && !block_table) ||
                         seq_len == cached_len || seq_len == new_len || cu_new == cached_len ||
                         cu_new == new_len))
    return MPZCH_EINVAL;
  TablesArgs a;
  a.cached = cached_len;
  a.news = new_len;
  a.B = n_requests;
  a.bs_log = log2_of(block_size);
  a.free_blocks = free_blocks;
  a.n_free = n_free_blocks;
  a.free_count = reinterpret_cast<const long long*>(free_count);
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.cu = cu_new;
  a.seq = seq_len;
  a.slots = reinterpret_cast<long long*>(slots);
  a.n_slots = n_slots;
  a.free_out = reinterpret_cast<long long*>(free_count_out);
  a.status = dev_status;
  const int block = n_requests <= 1024 ? 256 : 1024;
  const size_t smem = (size_t)n_requests * 2 * sizeof(int32_t);
  // 8 rows or requests a thread at least, one block an SM at most
  const int64_t work = (n_slots > n_requests ? n_slots : n_requests) / 8;
  return launch_smem(k_kv_tables, grid_for(work, block, 1), block, smem, S(stream), true, a);
}

int mpzch_kv_append(const void* k, int64_t k_stride_n, int64_t k_stride_h, const void* v,
                    int64_t v_stride_n, int64_t v_stride_h, int64_t n, int32_t dtype,
                    const int64_t* slots, int8_t* k_cache, int8_t* v_cache, float* k_scale,
                    float* v_scale, int64_t num_blocks, int32_t block_size, int32_t kv_heads,
                    int32_t dim, int32_t* dev_status, void* stream) {
  const int bytes = type_bytes(dtype);
  if (n < 0 || n > kMaxInt || bytes == 0 || !block_size_ok(block_size) || !dim_ok(dim) ||
      kv_heads < 1 || kv_heads > 4096 || num_blocks < 0 || num_blocks > kMaxInt)
    return MPZCH_EINVAL;
  if (n == 0) return MPZCH_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale ||
      !rows_ok(k, k_stride_n, k_stride_h, bytes) || !rows_ok(v, v_stride_n, v_stride_h, bytes) ||
      !aligned16(k_cache) || !aligned16(v_cache) || k_cache == v_cache || k_scale == v_scale)
    return MPZCH_EINVAL;
  AppendArgs a;
  a.x[0] = k;
  a.x[1] = v;
  a.sn[0] = k_stride_n;
  a.sn[1] = v_stride_n;
  a.sh[0] = k_stride_h;
  a.sh[1] = v_stride_h;
  a.n = n;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.num_blocks = num_blocks;
  a.bs_log = log2_of(block_size);
  a.H = kv_heads;
  a.status = dev_status;
  // as many rows a warp as leave 32 warps for every SM
  const int64_t want = (int64_t)sm_count() * 32;
  int64_t rpw = n * kv_heads * 2 / want;
  a.rows_per_warp = (int)(rpw < 1 ? 1 : rpw > 32 ? 32 : rpw);
  const cudaStream_t st = S(stream);
  return dtype == MPZCH_F32 ? launch_append_dim<float>(a, dim, st)
                            : dtype == MPZCH_F16 ? launch_append_dim<__half>(a, dim, st)
                                                 : launch_append_dim<__nv_bfloat16>(a, dim, st);
}

int64_t mpzch_kv_attend_workspace(int32_t q_heads, int32_t kv_heads, int32_t dim) {
  if (kv_heads < 1 || q_heads < 1 || q_heads > 4096 || q_heads % kv_heads || !dim_ok(dim)) return -1;
  return part_bytes(dim);
}

int mpzch_kv_attend(const void* q, int64_t q_stride_n, int64_t q_stride_h, int64_t n, int32_t dtype,
                    const int8_t* k_cache, const int8_t* v_cache, const float* k_scale,
                    const float* v_scale, int64_t num_blocks, int32_t block_size, int32_t q_heads,
                    int32_t kv_heads, int32_t dim, const int32_t* block_table, int32_t max_blocks,
                    const int32_t* cu_new, const int32_t* seq_len, int32_t n_requests,
                    int32_t max_new, float softmax_scale, int32_t causal, int32_t window, void* out,
                    int64_t out_stride_n, int64_t out_stride_h, float* lse, void* workspace,
                    int64_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int bytes = type_bytes(dtype);
  const int64_t need = mpzch_kv_attend_workspace(q_heads, kv_heads, dim);
  if (need < 0 || bytes == 0 || n < 0 || n > (kMaxInt - 1024) / q_heads || !block_size_ok(block_size) ||
      num_blocks < 0 || num_blocks > kMaxInt || max_blocks < 0 || n_requests < 0 ||
      n_requests > MPZCH_KV_MAX_REQUESTS || max_new < 0 ||
      !std::isfinite(softmax_scale * kLog2E) ||
      window < 0 || (window > 0 && !causal) ||
      ((int64_t)max_blocks * block_size > kMaxInt - 1024))
    return MPZCH_EINVAL;
  if (n == 0 || n_requests == 0) return MPZCH_OK;
  if (!q || !out || !cu_new || !seq_len || (max_blocks > 0 && !block_table) ||
      (num_blocks > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)) || !workspace ||
      workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      !rows_ok(q, q_stride_n, q_stride_h, bytes) || !rows_ok(out, out_stride_n, out_stride_h, bytes) ||
      !aligned16(k_cache) || !aligned16(v_cache))
    return MPZCH_EINVAL;
  if (heads_overlap(n, out_stride_n, q_heads, out_stride_h, dim)) return MPZCH_EINVAL;
  AttendArgs a;
  a.q = q;
  a.qsn = q_stride_n;
  a.qsh = q_stride_h;
  a.n = n;
  a.k = k_cache;
  a.v = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.num_blocks = num_blocks;
  a.bs_log = log2_of(block_size);
  a.Hq = q_heads;
  a.H = kv_heads;
  a.G = q_heads / kv_heads;
  a.table = block_table;
  a.max_blocks = max_blocks;
  a.cu = cu_new;
  a.seq = seq_len;
  a.B = n_requests;
  a.scale_log2 = softmax_scale * kLog2E;
  a.causal = causal ? 1 : 0;
  a.window = window;
  a.out = out;
  a.osn = out_stride_n;
  a.osh = out_stride_h;
  a.out_sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0 && out_stride_n * bytes % 32 == 0 &&
                  out_stride_h * bytes % 32 == 0;
  a.lse = lse;
  a.status = dev_status;
  const int64_t most = (int64_t)max_blocks * block_size;
  a.unit_keys = most <= kTinyKeys || (most <= kWholeKeys && (int64_t)a.B * a.H <= kWholeItems)
                    ? 1 << 30
                    : kUnitKeys;
  a.item_cost = a.unit_keys == kUnitKeys ? kRowItemCost : 0;
  a.max_new = max_new;
  a.heads = static_cast<PartHead*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + head_bytes());
  const cudaStream_t st = S(stream);
  return dtype == MPZCH_F32 ? launch_rows_dim<float, 2, 2>(a, dim, st)
                            : dtype == MPZCH_F16 ? launch_rows_dim<__half, 1, 2>(a, dim, st)
                                                 : launch_rows_dim<__nv_bfloat16, 1, 1>(a, dim, st);
}

}  // extern "C"
