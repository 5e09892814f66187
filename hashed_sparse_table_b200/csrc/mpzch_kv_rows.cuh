// Attention over the history cache for few rows per request (decode steps,
// drafted tokens), and for every shape the tile kernel does not take.
#pragma once
#include "mpzch_kv_kernels.cuh"

namespace mpzch_kv {

constexpr int kMaxRows = 16;    // query rows (token, head of the group) of a tile: 8 or 16
constexpr int kUnitKeys = 64;   // keys of one unit of work: four steps of a warp
constexpr int kStepKeys = 16;
constexpr int kRowItemCost = 1;  // queries, result and the empty ring, in units
constexpr int kRowWarps = 4;    // independent warps of a block
constexpr int kRowBlocksPerSm = 4;

struct AttendArgs {
  const void* q;
  int64_t qsn, qsh, n;
  const int8_t *k, *v;
  const float *ks, *vs;
  int64_t num_blocks;
  int bs_log, Hq, H, G;  // H kv heads, G = Hq / H
  const int32_t* table;
  int max_blocks;
  const int32_t *cu, *seq;
  int B;
  float scale_log2;  // softmax_scale * log2(e)
  int causal, window;
  void* out;
  int64_t osn, osh;
  int out_sectors;    // every head of out starts on a 32-byte boundary
  float* lse;
  int32_t* status;
  int unit_keys;      // keys of one unit of work: kUnitKeys, or all of an item
  int item_cost;      // units that the shares count for an item besides its keys
  int max_new;        // the caller's bound on a request's rows: sizes the join's grid
  struct PartHead* heads;
  float* parts;       // [warp][2]: [R][D] means over the part's keys, [R][2] maxima and sums
};

// What a warp of k_kv_rows leaves for k_kv_join: the item that begins in the
// warp's share and ends in that of warp `last` (< 0: none).
struct PartHead {
  int32_t b, h, tile, last;
};

// n * Hq < 2^31 (checked by the host), so rows and positions are ints.
struct Request {
  int start;  // first row of the batch
  int w;      // rows (new tokens)
  int L;      // keys
};

__device__ __forceinline__ Request request_of(const AttendArgs& a, int b, bool report) {
  Request r;
  const int s0 = a.cu[b], e0 = a.cu[b + 1], l0 = a.seq[b];
  const int n = (int)a.n, most = a.max_blocks << a.bs_log;
  const int s = min(max(s0, 0), n), e = min(max(e0, s), n), l = min(max(l0, 0), most);
  if (report && (s != s0 || e != e0 || l != l0)) set_status(a.status, kStBadLen);
  r.start = s;
  r.w = e - s;
  r.L = l;
  return r;
}

// First key inside the window of position p.
__device__ __forceinline__ int window_low(const AttendArgs& a, int p) {
  return a.window && p >= a.window ? p - a.window + 1 : 0;
}
// One behind the last key that position p sees.
__device__ __forceinline__ int causal_high(const AttendArgs& a, const Request& r, int p) {
  return a.causal ? max(0, min(r.L, p + 1)) : r.L;
}

// First key that any row of the request sees, rounded down to 16.
__device__ __forceinline__ int first_key(const AttendArgs& a, const Request& r) {
  return window_low(a, r.L - r.w) & ~15;
}

// Units of one (head, row tile) of the request; every such item has the same
// number, at least one.
__device__ __forceinline__ int item_units(const AttendArgs& a, const Request& r) {
  const int keys = r.L - first_key(a, r);
  return keys > a.unit_keys ? (keys + a.unit_keys - 1) / a.unit_keys : 1;
}

template <int R>
__device__ __forceinline__ int row_tiles(const AttendArgs& a, const Request& r) {
  return (r.w * a.G + R - 1) / R;
}

template <int R>
__device__ __forceinline__ long long request_units(const AttendArgs& a, const Request& r) {
  return (long long)(row_tiles<R>(a, r) * a.H) * (item_units(a, r) + a.item_cost);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 x 8 matrix of fp16, a row to four lanes, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Codes (biased by 128) of bytes `sel` of x as two fp16 numbers: 0x6400 | u is
// 1024 + u exactly, and 1152 = 1024 + 128 comes off exactly.
__device__ __forceinline__ uint32_t codes_half2(uint32_t biased, uint32_t sel) {
  const uint32_t m = __byte_perm(biased, 0x64646464u, sel);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(0x64806480u));
  return r;
}
constexpr uint32_t kSelLow = 0x4140, kSelHigh = 0x4342;

template <int kWords>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
  if constexpr (kWords == 4) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  } else if constexpr (kWords == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const int8_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Byte of 16-byte chunk `col` of row `row` in a staged 16 x D tile.  The rows lie
// one behind the other; chunks change places within a 128-byte line so that the
// lanes of one shared-memory phase hit different banks:
//  keys, D = 128: lanes (row r, chunk c) of two rows r, r + 1 meet: bit 2 by r's parity
//  values: lanes (row 2c, chunk of r) of four even (or odd) rows meet.
template <int D, bool kValue>
__device__ __forceinline__ int staged(int row, int col) {
  const int at = row * (D / 16) + col, line = at >> 3, p = at & 7;
  if constexpr (!kValue)
    return D == 128 ? line * 128 + ((p ^ ((row & 1) << 2)) << 4) : at << 4;
  const int x = D == 128 ? row & 7 : D == 64 ? (2 * line) & 7 : (2 * line) & 2;
  return line * 128 + ((p ^ x) << 4);
}

// 4 consecutive query values as fp32.
template <typename T>
__device__ __forceinline__ void load4(const T* p, float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)h[i];
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    T h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = (T)x[i];
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(h);
  }
}

// Power of two that brings a row's largest |q| into [2^13, 2^14); NaN for a row
// that holds a NaN or an infinity, so that its scores are NaN.
__device__ __forceinline__ float row_factor(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  int e = 13 + 127 - (int)(amax_bits >> 23);  // exponent of the factor
  e = e > 100 ? 100 : e < -120 ? -120 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The softmax weights are kept as p * value scale * 2^7 / 2^ev in fp16.  A row's ev follows
// the largest product p * value scale that it has met, as the maximum follows its scores:
// both move only when a key passes them by more than kSlack, so the largest weight is 2^15;
// weights below 2^-21 of the row's largest lose bits and those below 2^-32 vanish, whatever
// the scales of blocks that the row does not look at.  Lower bounds of ev (kLeastRef, and
// kFar below the largest scale of any block so far) keep 2^7 / 2^ev and its product with a
// scale finite.
constexpr float kSlack = 8.f;
constexpr float kLeastRef = -119.f, kMostRef = 128.f, kFar = 100.f;
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e, e a whole number from -126 to 127.
__device__ __forceinline__ float exp2_whole(float e) {
  return __int_as_float(((int)e + 127) << 23);
}
// A finite value scale above all so far: the power of two above it, and the bound of ev.
__device__ __forceinline__ void raise_top(float va, float& vtop, float& least) {
  const int e = min(254, (int)(__float_as_uint(va) >> 23) + 1);
  vtop = __int_as_float(e << 23);
  least = fmaxf(kLeastRef, (float)(e - 127) - kFar);
}
// A row's ev for the largest product 2^d.
__device__ __forceinline__ float row_ref(float d, float least) {
  return fminf(fmaxf(ceilf(d), least), kMostRef);
}

// 16-key slots of a warp's ring: one being read, the others in flight.  12 KB a warp
// at D = 128: 12 warps of an SM have 96 KB under way.  (256 single tokens x 8 heads x
// 128: 108 us; four slots 110 us, 8 or 16 warps an SM 110 and 112 us.)
__host__ __device__ constexpr int row_slots(int D) { return D == 128 ? 3 : D == 64 ? 5 : 8; }
__host__ __device__ constexpr int row_smem(int D) { return kRowWarps * row_slots(D) * 2 * kStepKeys * D; }

// Writes D / 8 consecutive outputs.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* p, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float y[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
    store4<T>(p + i, y);
  }
}

// Single tokens and other few rows.  Every warp is a worker of its own: the units
// (64 keys of one request, kv head and row tile) of the whole batch are laid in a
// row and each warp takes an equal share of them, so ragged histories balance
// without the host knowing a length.  An item that two shares cut leaves parts for
// k_kv_join.  A warp works 16 keys of one block at a time while cp.async brings the
// next ones (a ring per warp, no block-wide barrier).  Products are m16n8k16 in fp16,
// the codes turned into fp16 in registers as operand A (16 rows of it), the few query
// rows as the 8-wide operand B:
//   scores   S^T = K Q^T      A: 16 keys x 16 dims
//   outputs  O^T = V^T P^T    A: 16 dims x 16 keys; P^T is S^T's lanes transposed
//                             (movmatrix on pairs of fp16)
// so 8 rows need half of what a 16-row tile of queries as A would.  Dims and keys are
// assigned to lanes so that no code changes lanes: for keys, lane (r, c) holds chunks c
// of keys r and r + 8 (dims in the same order for the queries); for values it holds
// keys 2c, 2c+1, 2c+8, 2c+9 and D / 8 neighbouring dims, two to each 16-dim tile.
// Bound by HBM and, close behind, by issuing about 450 instructions for 4 KB of codes
// (turning a byte into fp16 is one byte permutation and one subtraction for two): 256
// tokens, 32 query and 8 kv heads x 128, 515 MB of cache, 110 us with the join, 4.7 TB/s,
// 0.72 of the measured copy rate; two histories of 78 and 110 thousand keys, 4 kv heads x
// 128, fp16, 193 MB, 49 us; 4,096 fp32 histories of up to 1,000 keys, 4 heads x 128, 625 MB,
// 204 us (two products for each, and half of the time in beginning and ending items).
template <int D, typename T, int R, int NQ, int NP>
__global__ void __launch_bounds__(32 * kRowWarps, R == 8 ? (D == 128 ? 3 : 4) : NQ == 1 ? 3 : 2)
    k_kv_rows(AttendArgs a) {
  pdl_enter();
  constexpr int kWK = D >= 64 ? 4 : 2;       // words per load of key bytes
  constexpr int kChunks = D >= 64 ? D / 64 : 1;
  constexpr int kK = kWK * kChunks;          // key words a lane holds per key = MMA k-steps
  constexpr int kWV = D / 32;                // value words a lane holds per key
  constexpr int kTile = kStepKeys * D;       // bytes of a staged tile
  constexpr int kCols = D / 16;
  constexpr int kSlots = row_slots(D);
  constexpr int NR = R / 8;                  // rows of a lane
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ long long s_sum[kRowWarps];
  __shared__ long long s_upto[32 * kRowWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int worker = blockIdx.x * kRowWarps + warp;
  const int bs = 1 << a.bs_log;
  pdl_trigger();  // the join's blocks may take their places; they wait for this grid

  // ---- this warp's share of the units of all items
  const int per_thread = (a.B + blockDim.x - 1) / blockDim.x;
  {
    const int b_lo = tid * per_thread, b_hi = min(a.B, b_lo + per_thread);
    long long upto = 0;
    for (int b = b_lo; b < b_hi; ++b)
      upto += request_units<R>(a, request_of(a, b, blockIdx.x == 0));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(kAll, upto, d);
      if (lane >= d) upto += y;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    for (int i = 0; i < warp; ++i) upto += s_sum[i];
    s_upto[tid] = upto;
    __syncthreads();
  }
  const long long total = s_upto[32 * kRowWarps - 1];
  const long long workers = (long long)gridDim.x * kRowWarps;
  long long per = (total + workers - 1) / workers;
  if (per < 1) per = 1;
  long long u = per * worker;
  const long long u_end = min(total, u + per);
  PartHead head = {0, 0, 0, -1};
  if (u >= u_end) {
    if (lane == 0) a.heads[worker] = head;
    return;
  }
  int b = 0;
  long long b_units = 0;  // units before request b
  {
    int first = 0;  // threads whose requests end at or before u
    for (int i = 0; i < kRowWarps; ++i)
      first += __popc(__ballot_sync(kAll, s_upto[i * 32 + lane] <= u));
    b = first * per_thread;
    b_units = first ? s_upto[first - 1] : 0;
    // 32 requests at a time
    for (;;) {
      const int mine = b + lane;
      long long x = mine < a.B ? request_units<R>(a, request_of(a, mine, false)) : 0, upto = x;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(kAll, upto, d);
        if (lane >= d) upto += y;
      }
      const int past = __popc(__ballot_sync(kAll, b_units + upto <= u));
      if (past < 32) {
        if (past) b_units += __shfl_sync(kAll, upto, past - 1);
        b += past;
        break;
      }
      b_units += __shfl_sync(kAll, upto, 31);
      b += 32;
    }
  }
  const uint32_t ring =
      (uint32_t)__cvta_generic_to_shared(s_ring) + warp * (kSlots * 2 * kTile);

  // Where this lane's chunks go in a staged tile, and where it reads: staged() taken
  // apart, so that the loop adds one of a few numbers to a slot's address.  Key chunk 1
  // (D = 128) lies at the flipped bit 6; value rows 2c + 1 at v_at1, rows 8 on 8 rows on;
  // value chunks of every other group of 4 rows at the flipped bit 6 too.
  constexpr uint32_t kOdd = D == 128 ? 64 : 0;
  const uint32_t k_to = staged<D, false>(lane / kCols, lane % kCols);
  const uint32_t v_to = staged<D, true>(lane / kCols, lane % kCols);
  const uint32_t k_at = D >= 64 ? staged<D, false>(r, c) : r * D + c * 8;
  const uint32_t v_at0 = staged<D, true>(2 * c, r * (D / 8) >> 4) + (r * (D / 8) & 15);
  const uint32_t v_at1 = staged<D, true>(2 * c + 1, r * (D / 8) >> 4) + (r * (D / 8) & 15);

  while (u < u_end) {
    const Request req = request_of(a, b, false);
    const int tiles = row_tiles<R>(a, req), units = item_units(a, req);
    const int cost = units + a.item_cost;
    const long long all = (long long)(tiles * a.H) * cost;
    if (b_units + all <= u) {
      b_units += all;
      ++b;
      continue;
    }
    const long long into = u - b_units;
    const int item = (into >> 32) ? (int)(into / cost) : (int)((uint32_t)into / (uint32_t)cost);
    // the share takes [x0, x1) of the item's cost, which are its units [u0, u1); one that
    // ends before the first unit leaves the item to the next share
    const int x0 = (int)(into - (long long)item * cost);
    const int x1 = (int)min((long long)cost, x0 + (u_end - u));
    const int u0 = max(0, x0 - a.item_cost), u1 = max(0, x1 - a.item_cost);
    if (u0 == u1) break;
    const int h = item / tiles, tile = item % tiles;
    const int rows = req.w * a.G, first_row = tile * R;
    const int n_rows = min(R, rows - first_row);

    // ---- keys that any row of the tile sees, and keys that all of them see; the
    // steps of this share among the former
    const int p_lo = req.L - req.w + first_row / a.G;
    const int p_hi = req.L - req.w + (first_row + n_rows - 1) / a.G;
    const int any_hi = causal_high(a, req, p_hi), any_lo = window_low(a, p_lo);
    const int all_hi = causal_high(a, req, p_lo), all_lo = window_low(a, p_hi);
    const int key0 = first_key(a, req);
    const int k_lo = max(key0 + u0 * a.unit_keys, any_lo & ~15);
    const int k_hi = (int)min((long long)any_hi, key0 + (long long)u1 * a.unit_keys);
    const int n_steps = k_hi > k_lo ? (k_hi - k_lo + kStepKeys - 1) / kStepKeys : 0;

    // Block id and scales of step 32 g + lane: group `c` of the steps that are
    // computed and the next one, `n`.
    int32_t id_c, id_n;
    float ks_c, vs_c, ks_n, vs_n;
    const int32_t* row_table = a.table + (int64_t)b * a.max_blocks;
    auto look_up = [&](int s, int32_t& id, float& ks, float& vs) {
      id = -1;
      ks = vs = 0.f;
      if (s < n_steps) {
        id = __ldg(row_table + ((k_lo + s * kStepKeys) >> a.bs_log));
        if (id < 0 || id >= a.num_blocks) {
          id = -1;
          set_status(a.status, kStBadBlock);
        } else {
          ks = __ldg(a.ks + (int64_t)id * a.H + h);
          vs = __ldg(a.vs + (int64_t)id * a.H + h);
        }
      }
    };
    // this lane's chunks of head h: chunk i * 32 + lane of a tile
    const int8_t* kb = a.k + ((int64_t)h << a.bs_log) * D + lane * 16;
    const int8_t* vb = a.v + ((int64_t)h << a.bs_log) * D + lane * 16;
    const int block_bytes = (a.H << a.bs_log) * D;
    auto fetch = [&](int s, int32_t id, uint32_t to) {  // id: of step s, -1 for none
      if (id >= 0) {
        const int64_t off =
            (int64_t)id * block_bytes + ((k_lo + s * kStepKeys) & (bs - 1)) * D;
#pragma unroll
        for (int i = 0; i < kTile / 512; ++i) {
          copy16(to + k_to + i * 512, kb + off + i * 512);
          copy16(to + kTile + (i & 1 ? v_to ^ kOdd : v_to) + i * 512, vb + off + i * 512);
        }
      }
      copies_commit();
    };
    look_up(lane, id_c, ks_c, vs_c);
#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s)
      fetch(s, __shfl_sync(kAll, id_c, s), ring + s * (2 * kTile));
    look_up(32 + lane, id_n, ks_n, vs_n);
    uint32_t slot = ring, free_slot = ring + (kSlots - 1) * (2 * kTile);

    // ---- the tile's query rows
    // B operands: lane (r, c) holds row 8 i + r.  Factors, limits, maxima and sums
    // are kept where the results are: rows 8 i + 2c + k, index [i][k].
    float inv[NR][2];
    int row_hi[NR][2], row_lo[NR][2];
    uint32_t qf[NQ][NR][kK][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = first_row + r + 8 * i;
      const bool real = row < rows;
      const int t = real ? row / a.G : 0;
      const T* p = static_cast<const T*>(a.q) + (req.start + t) * a.qsn +
                   (h * a.G + (real ? row - t * a.G : 0)) * a.qsh;
      float x[kK][4];
      uint32_t amax = 0;
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        const int d = D >= 64 ? (kk / 4) * 64 + c * 16 + (kk % 4) * 4 : c * 8 + kk * 4;
        if (real) {
          load4<T>(p + d, x[kk]);
        } else {
          x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max(amax, __float_as_uint(x[kk][e]) & 0x7FFFFFFFu);
      }
      amax = max(amax, __shfl_xor_sync(kAll, amax, 1));
      amax = max(amax, __shfl_xor_sync(kAll, amax, 2));
      // a negative softmax scale goes into the sign of the query
      const float f = copysignf(row_factor(amax), a.scale_log2);
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = f != f ? 0.f : __fmul_rn(x[kk][e], f);
        qf[0][i][kk][0] = half2_bits(y[0], y[1]);
        qf[0][i][kk][1] = half2_bits(y[2], y[3]);
        if constexpr (NQ == 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = __fsub_rn(y[e], __half2float(__float2half_rn(y[e])));
          qf[NQ - 1][i][kk][0] = half2_bits(y[0], y[1]);
          qf[NQ - 1][i][kk][1] = half2_bits(y[2], y[3]);
        }
      }
      const int pos = req.L - req.w + t;
      const float own = __fdiv_rn(a.scale_log2, f);
      const int hi = real ? causal_high(a, req, pos) : 0;
      const int lo = window_low(a, pos);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        inv[i][k] = __shfl_sync(kAll, own, 8 * c + 4 * k);
        row_hi[i][k] = __shfl_sync(kAll, hi, 8 * c + 4 * k);
        row_lo[i][k] = __shfl_sync(kAll, lo, 8 * c + 4 * k);
      }
    }

    // acc[i][t]: rows 8 i + 2c, 8 i + 2c + 1 of the lane's dims 2t, then of 2t + 1
    float acc[NR][D / 16][4];
    float m[NR][2], l[NR][2];  // running maxima (log2 units), sums over this lane's keys
    float d[NR][2];            // log2 of the largest p * value scale, and kSlack
    float wt[NR][2];           // 2^7 / 2^ev
    float vtop = 0.f, least = kLeastRef;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i][0] = m[i][1] = -CUDART_INF_F;
      l[i][0] = l[i][1] = 0.f;
      d[i][0] = d[i][1] = -CUDART_INF_F;
      wt[i][0] = wt[i][1] = 1.f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) acc[i][t][0] = acc[i][t][1] = acc[i][t][2] = acc[i][t][3] = 0.f;
    }

    for (int s = 0; s < n_steps; ++s) {
      const int at = s & 31;
      if (at == 0 && s) {
        id_c = id_n;
        ks_c = ks_n;
        vs_c = vs_n;
        look_up(s + 32 + lane, id_n, ks_n, vs_n);
      }
      copies_wait<kSlots - 2>();
      __syncwarp();  // every lane's copies of step s have landed, step s - 1 is read
      fetch(s + kSlots - 1,
            __shfl_sync(kAll, at + kSlots - 1 < 32 ? id_c : id_n, (s + kSlots - 1) & 31), free_slot);
      const uint32_t kt = slot, vt = slot + kTile;
      free_slot = slot;
      slot = slot + 2 * kTile == ring + kSlots * 2 * kTile ? ring : slot + 2 * kTile;
      const int32_t id = __shfl_sync(kAll, id_c, at);
      float ks = __shfl_sync(kAll, ks_c, at);
      const float vs = __shfl_sync(kAll, vs_c, at);
      if (id < 0) continue;  // a block outside the cache
      const int key = k_lo + s * kStepKeys;

      uint32_t kw[2][kK];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          lds_words<kWK>(kt + (i ? k_at ^ 64 : k_at) + j * 8 * D, &kw[j][i * kWK]);
      }
      uint32_t vw[4][kWV];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lds_words<kWV>(vt + (j & 1 ? v_at1 : v_at0) + (j >> 1) * 8 * D, vw[j]);
      }
      float sc[NR][4];  // [rows 8 i ..][2 j + k]: key r + 8 j, row 2c + k
#pragma unroll
      for (int i = 0; i < NR; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        const uint32_t x0 = kw[0][kk] ^ 0x80808080u, x1 = kw[1][kk] ^ 0x80808080u;
        const uint32_t ka[4] = {codes_half2(x0, kSelLow), codes_half2(x1, kSelLow),
                                codes_half2(x0, kSelHigh), codes_half2(x1, kSelHigh)};
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int t = 0; t < NQ; ++t) mma_16816(sc[i], ka, qf[t][i][kk][0], qf[t][i][kk][1]);
      }
      const bool hide = key + kStepKeys > all_hi || key < all_lo;
      uint32_t hidden = 0;  // bit i * 4 + 2 j + k
      if (hide) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = key + r + 8 * (e >> 1);
            if (k >= row_hi[i][e & 1] || k < row_lo[i][e & 1]) {
              sc[i][e] = -CUDART_INF_F;
              hidden |= 1u << (i * 4 + e);
            }
          }
      }
      if (ks < 0.f) {  // no append gives one
        ks = -ks;
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!(hidden >> (i * 4 + e) & 1)) sc[i][e] = -sc[i][e];
      }
      float f[NR][2], mx[NR][2];
      bool up = false;
      const float va = fabsf(vs), lva = log2_fast(va);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          f[i][k] = __fmul_rn(inv[i][k], ks);
          mx[i][k] = fmaxf(sc[i][k], sc[i][k + 2]);
          mx[i][k] = mx[i][k] == -CUDART_INF_F ? mx[i][k] : __fmul_rn(mx[i][k], f[i][k]);
          const float x = mx[i][k] - m[i][k];  // NaN where nothing has been seen: not up
          up |= x > kSlack || x + lva > d[i][k];
        }
      const bool vup = va > vtop && va < CUDART_INF_F;
      if (__any_sync(kAll, up || vup)) {
        if (vup) raise_top(va, vtop, least);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          float g[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = mx[i][k];
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 16));
            const float to = fmaxf(m[i][k], x);
            const float alpha = to == m[i][k] ? 1.f : exp2_fast(m[i][k] - to);
            if (to != m[i][k]) d[i][k] += m[i][k] - to;
            d[i][k] = fmaxf(d[i][k], x - to + (lva + kSlack));
            m[i][k] = to;
            l[i][k] = __fmul_rn(l[i][k], alpha);
            const float w = exp2_whole(7.f - row_ref(d[i][k] - kSlack, least));
            g[k] = __fmul_rn(alpha, __fdiv_rn(w, wt[i][k]));
            wt[i][k] = w;
          }
#pragma unroll
          for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][t][e] = __fmul_rn(acc[i][t][e], g[e & 1]);
        }
      }
      uint32_t pb[NP][NR][2];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float base = m[i][e & 1] == -CUDART_INF_F ? 0.f : m[i][e & 1];
          // rounded like the maximum, so that the largest score gives 2^0 at any size
          p[e] = exp2_fast(__fsub_rn(__fmul_rn(sc[i][e], f[i][e & 1]), base));
          if (hide && (hidden >> (i * 4 + e) & 1)) p[e] = 0.f;
        }
        l[i][0] = __fadd_rn(l[i][0], __fadd_rn(p[0], p[2]));
        l[i][1] = __fadd_rn(l[i][1], __fadd_rn(p[1], p[3]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = __fmul_rn(p[e], __fmul_rn(wt[i][e & 1], vs));
          // weight 0 whatever the block's scale is
          if (hide && (hidden >> (i * 4 + e) & 1)) p[e] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < NP; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            pb[t][i][j] = transposed(half2_bits(p[2 * j], p[2 * j + 1]));
            if (t + 1 < NP) {
              p[2 * j] = __fsub_rn(p[2 * j], __half2float(__float2half_rn(p[2 * j])));
              p[2 * j + 1] = __fsub_rn(p[2 * j + 1], __half2float(__float2half_rn(p[2 * j + 1])));
            }
          }
      }
#pragma unroll
      for (int w = 0; w < kWV; ++w) {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = vw[j][w] ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // dims 4w + 2e, 4w + 2e + 1 of the lane
          const uint32_t sel = e ? 0x7362 : 0x5140;
          const uint32_t near = __byte_perm(x[0], x[1], sel), far = __byte_perm(x[2], x[3], sel);
          const uint32_t va4[4] = {codes_half2(near, kSelLow), codes_half2(near, kSelHigh),
                                   codes_half2(far, kSelLow), codes_half2(far, kSelHigh)};
#pragma unroll
          for (int i = 0; i < NR; ++i)
#pragma unroll
            for (int t = 0; t < NP; ++t)
              mma_16816(acc[i][w * 2 + e], va4, pb[t][i][0], pb[t][i][1]);
        }
      }
    }
    copies_wait<0>();
    __syncwarp();  // the ring is free for the next item

    // ---- results: lane (r, c) holds dims r * D / 8 .. of rows 8 i + 2c + j
    const bool begins = u0 == 0, ends = u1 == units;
    const bool whole = begins && ends;
    float* part = a.parts + ((int64_t)worker * 2 + (begins ? 1 : 0)) * R * (D + 2);
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * i + 2 * c + j;
        const float top = m[i][j];
        float L = l[i][j];
        L += __shfl_xor_sync(kAll, L, 4);
        L += __shfl_xor_sync(kAll, L, 8);
        L += __shfl_xor_sync(kAll, L, 16);
        if (row >= n_rows) continue;
        // the mean, also of a part (sums of large values would overflow), in two steps, since
        // 1 / (wt L) can underflow; a row that saw no key has an all-zero accumulator
        const float unit = __fdiv_rn(1.f, wt[i][j]);
        const float g = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
        const int at = first_row + row, t = at / a.G;
        const int hq = h * a.G + at - t * a.G;
        float o[D / 8];
#pragma unroll
        for (int k = 0; k < D / 8; ++k) o[k] = __fmul_rn(__fmul_rn(acc[i][k / 2][2 * (k & 1) + j], g), unit);
        const int d = r * (D / 8);
        if (whole) {
          store_row<T>(static_cast<T*>(a.out) + (req.start + t) * a.osn + hq * a.osh + d, o);
          if (a.lse && r == 0)
            a.lse[(int64_t)(req.start + t) * a.Hq + hq] =
                L == 0.f ? -CUDART_INF_F : __fmul_rn(top + log2f(L), 0.6931471805599453f);
        } else {
          store_row<float>(part + row * D + d, o);
          if (r == 0) *reinterpret_cast<float2*>(part + R * D + row * 2) = make_float2(top, L);
        }
      }
    }
    if (begins && !ends) {
      head.b = b;
      head.h = h;
      head.tile = tile;
      head.last = (int)((b_units + (item + 1ll) * cost - 1) / per);
    }
    u += x1 - x0;
  }
  if (lane == 0) a.heads[worker] = head;
}

// Joins the parts of the items that k_kv_rows or k_kv_tiles split: an item that begins in
// worker i's share and goes on into the next ones.  A block (x, .) looks after
// kJoinHeads workers.  Items of few parts are joined a row to a warp; those of many a row
// to a block (the y-th block of x takes rows y, y + gridDim.y, ..), whose warps take every
// kJoinWarps-th part.  The weights of all parts come first (one load a lane), so the
// parts' loads do not wait for one another.  All sums have a fixed order.
constexpr int kJoinWarps = 8, kFewParts = 32, kMostParts = 2368;
template <int R>
__host__ __device__ constexpr int join_heads() { return R > 16 ? 1 : 4; }

template <int D, typename T, int R>
struct Join {
  static constexpr int kPer = D / 32, kRound = 4;
  static constexpr int64_t kPart = (int64_t)R * (D + 2);
  const AttendArgs& a;
  PartHead head;
  const float* all;  // of the worker that begins the item
  int parts, row, lane;

  __device__ __forceinline__ Join(const AttendArgs& args, int first, const PartHead& h)
      : a(args), head(h), all(args.parts + (int64_t)first * 2 * kPart), parts(h.last - first + 1),
        row(0), lane(threadIdx.x & 31) {}
  // part i: the first one is what its worker began, the others what theirs go on with
  __device__ __forceinline__ const float* part(int i) const {
    return all + (i ? (int64_t)i * 2 : 1) * kPart;
  }
  __device__ __forceinline__ float2 ml(int i) const {
    return *reinterpret_cast<const float2*>(part(i) + R * D + row * 2);
  }
  // a part's share of the sum; a part without a key has l = 0, one of NaN alone m = -inf
  __device__ __forceinline__ static float sum_of(float2 x, float M) {
    return x.y == 0.f ? 0.f : x.x == -CUDART_INF_F ? x.y : __fmul_rn(x.y, exp2_fast(x.x - M));
  }
  __device__ __forceinline__ bool real(const Request& req) const {
    return head.tile * R + row < req.w * a.G;
  }
  // parts from, from + step, ..; weights, which add up to 1, by w(i)
  template <typename W>
  __device__ __forceinline__ void add(int from, int step, W w, float (&o)[kPer]) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = 0.f;
    for (int i0 = from; i0 < parts; i0 += step * kRound) {
      float x[kRound][kPer], e[kRound];
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        const int i = i0 + j * step;
        e[j] = w(i);  // (the whole warp: it may be a shuffle)
        if (i < parts) {
          const float* p = part(i) + row * D + lane;
#pragma unroll
          for (int k = 0; k < kPer; ++k) x[j][k] = p[32 * k];
        } else {
          e[j] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < kRound; ++j)
#pragma unroll
        for (int k = 0; k < kPer; ++k)
          if (e[j] != 0.f) o[k] = __fmaf_rn(x[j][k], e[j], o[k]);
    }
  }
  __device__ __forceinline__ void store(const Request& req, const float (&o)[kPer], float M,
                                        float L) const {
    const int at = head.tile * R + row, t = at / a.G;
    const int hq = head.h * a.G + at - t * a.G;
    T* out = static_cast<T*>(a.out) + (req.start + t) * a.osn + hq * a.osh;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      out[lane + 32 * k] = (T)(L == 0.f ? 0.f : o[k]);
    if (a.lse && lane == 0)
      a.lse[(int64_t)(req.start + t) * a.Hq + hq] =
          L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
  }
};

template <int D, typename T, int R>
__global__ void __launch_bounds__(32 * kJoinWarps, 4) k_kv_join(AttendArgs a, int workers) {
  pdl_enter();
  constexpr int kHeads = join_heads<R>();
  __shared__ float s_w[kMostParts];       // weights of many parts
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float s_r[2][kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first0 = blockIdx.x * kHeads;
  for (int task = blockIdx.y * kJoinWarps + warp; task < kHeads * R; task += gridDim.y * kJoinWarps) {
    const int first = first0 + task / R;
    if (first >= workers) break;
    const PartHead head = a.heads[first];
    if (head.last < 0 || head.last - first >= kFewParts) continue;
    Join<D, T, R> join(a, first, head);
    join.row = task % R;
    const Request req = request_of(a, head.b, false);
    if (!join.real(req)) continue;
    const float2 ml = lane < join.parts ? join.ml(lane) : make_float2(-CUDART_INF_F, 0.f);
    float M = ml.x;
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, d));
    const float mine = join.sum_of(ml, M);
    float L = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) L = __fadd_rn(L, __shfl_xor_sync(kAll, L, d));
    const float weight = __fdiv_rn(mine, L);  // (all 0 / 0: not used)
    float o[D / 32];
    join.add(0, 1, [&](int i) { return __shfl_sync(kAll, weight, i & 31); }, o);
    join.store(req, o, M, L);
  }
  for (int n = 0; n < kHeads; ++n) {
    const int first = first0 + n;
    if (first >= workers) break;
    const PartHead head = a.heads[first];
    if (head.last < 0 || head.last - first < kFewParts) continue;
    Join<D, T, R> join(a, first, head);
    const Request req = request_of(a, head.b, false);
    for (join.row = blockIdx.y; join.row < R && join.real(req); join.row += gridDim.y) {
      float M = -CUDART_INF_F, L = 0.f;
      for (int i = threadIdx.x; i < join.parts; i += 32 * kJoinWarps) {
        s_w[i] = join.ml(i).x;
        M = fmaxf(M, s_w[i]);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, d));
      if (lane == 0) s_r[0][warp] = M;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_r[0][w]);
      for (int i = threadIdx.x; i < join.parts; i += 32 * kJoinWarps) {
        s_w[i] = join.sum_of(make_float2(s_w[i], join.ml(i).y), M);
        L = __fadd_rn(L, s_w[i]);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) L = __fadd_rn(L, __shfl_xor_sync(kAll, L, d));
      if (lane == 0) s_r[1][warp] = L;
      __syncthreads();
      L = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) L = __fadd_rn(L, s_r[1][w]);
      const float inv = __fdiv_rn(1.f, L);
      float o[D / 32];
      join.add(warp, kJoinWarps,
               [&](int i) { return i < join.parts ? __fmul_rn(s_w[i], inv) : 0.f; }, o);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) s_o[warp][lane + 32 * k] = o[k];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
#pragma unroll
          for (int w = 1; w < kJoinWarps; ++w) o[k] = __fadd_rn(o[k], s_o[w][lane + 32 * k]);
        join.store(req, o, M, L);
      }
      __syncthreads();  // the arrays are free for the next row
    }
  }
}

}  // namespace mpzch_kv
