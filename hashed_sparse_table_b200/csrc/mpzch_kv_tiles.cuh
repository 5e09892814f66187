// Attention over the history cache for many rows per request (admissions, chunks,
// candidates): 256-row tiles on the tensor cores (tcgen05, accumulators in TMEM).
#pragma once
#include "mpzch_kv_rows.cuh"

namespace mpzch_kv {

constexpr int kTileRows = 256;   // two halves of 128, each with its softmax warpgroup
constexpr int kTileKeys = 128;   // keys of one step
constexpr int kGroups = kTileKeys / 16;
constexpr int kSoftWarps = 16, kConvWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kConvWarps, kLoadWarp = kMmaWarp + 1;
constexpr int kTileThreads = 32 * (kLoadWarp + 1);
constexpr int kItems = 4;        // items known ahead
constexpr int kTileStages = 2;
constexpr int kScaleSlots = 4;
constexpr int kRawKeys = 64;     // keys of a raw slot; in turn K low, K high, V low, V high
constexpr int kRawSlots = 3;

// Shared memory: Q [2 halves][D / 64][128 rows][128 B], K and V stages
// [D / 64][128 keys][128 B], all in the 128-byte swizzle; then the codes as they come,
// [slot][64 keys][D], and the small fields.
template <int D>
struct TileSmem {
  static constexpr int kPlane = 128 * 128;            // 64 dims of 128 rows
  static constexpr int kOperand = D / 64 * kPlane;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kOperand;
  static constexpr int kV = kK + kTileStages * kOperand;
  static constexpr int kRaw = kV + kTileStages * kOperand;
  static constexpr int kSmall = kRaw + kRawSlots * kRawKeys * D;
  static constexpr int kBytes = kSmall + 8192 + 1024;  // and up to 1 KB to align the base
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy_bulk(uint32_t to, const void* from, uint32_t bytes, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
      "l"(from), "r"(bytes), "r"(smem_addr(b))
      : "memory");
}
// Waits for a phase; gives up after kWaitLimitNs (then, and once any warp of the
// block gave up, false).
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, volatile int32_t* failed,
                                         int32_t* status) {
  if (bar_test(b, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_test(b, parity)) return true;
    if (*failed) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *failed = 1;
      set_status(status, kStTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t leader, uint64_t* b) {
  asm volatile(
      "{\n.reg .pred q;\nsetp.ne.u32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_addr(b)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Operand descriptor, 128-byte swizzle: start address, leading and stride offsets in
// 16-byte units, version 1.  The low word moves with the address alone (shared memory
// ends below 2^18), so the issuing thread spends one addition for each operand.
__device__ __forceinline__ uint32_t operand_low(uint32_t addr, uint32_t lead) {
  return addr >> 4 | (lead >> 4) << 16;
}
__host__ __device__ constexpr uint32_t operand_high(uint32_t stride) { return stride >> 4 | 1u << 14 | 2u << 29; }
// fp16 x fp16 (bf16 x bf16) -> fp32, M = 128, N columns; B's N index contiguous if
// kTransposed.
template <int N, bool kTransposed, bool kBf16>
__device__ __forceinline__ constexpr uint32_t instruction() {
  return 1u << 4 | (kBf16 ? 1u << 7 | 1u << 10 : 0u) | (kTransposed ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}
// Issued by the warp's leader alone, under a predicate: the operands are the same in
// every lane, so they stay in uniform registers, which a branch for one lane would
// fill anew for each product (measured: 130 cycles a product instead of the 64 that it
// takes).
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t high, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 x, y;\nsetp.ne.u32 p, %5, 0;\nsetp.ne.u32 q, %6, 0;\n"
      "mov.b64 x, {%1, %3};\nmov.b64 y, {%2, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(idesc), "r"((uint32_t)add), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t high, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 y;\nsetp.ne.u32 p, %5, 0;\nsetp.ne.u32 q, %6, 0;\n"
      "mov.b64 y, {%2, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(high), "r"(idesc), "r"((uint32_t)add), "r"(leader)
      : "memory");
}

#define MPZCH_R8(x, i) \
  "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), \
      "=r"(x[i + 6]), "=r"(x[i + 7])
#define MPZCH_U8(x, i) \
  "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), \
      "r"(x[i + 6]), "r"(x[i + 7])
// 32 (16) neighbouring 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MPZCH_R8(x, 0), MPZCH_R8(x, 8), MPZCH_R8(x, 16), MPZCH_R8(x, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::MPZCH_U8(x, 0),
      MPZCH_U8(x, 8), MPZCH_U8(x, 16), MPZCH_U8(x, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15};" ::MPZCH_U8(x, 0),
      MPZCH_U8(x, 8), "r"(addr)
      : "memory");
}
#undef MPZCH_R8
#undef MPZCH_U8
// The loaded registers are valid behind this; they pass through it so that no use moves ahead.
__device__ __forceinline__ void tmem_loaded(uint32_t (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(x[i]));
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Bits of the keys k0 .. k0 + 31 that lie in [lo, hi).
__device__ __forceinline__ uint32_t keys_between(int k0, int lo, int hi) {
  const int from = max(0, lo - k0), to = min(32, hi - k0);
  if (to <= from || from > 31) return 0;
  return (to == 32 ? kAll : (1u << to) - 1) & ~((1u << from) - 1);
}

// Keys [lo, hi) that any row of the row tile sees, lo rounded down to 16, and the
// tile's steps (at least one).
struct TileRange {
  int lo, hi, steps;
};
__device__ __forceinline__ TileRange tile_range(const AttendArgs& a, const Request& r, int tile) {
  const int row0 = tile * kTileRows, row1 = min(row0 + kTileRows, r.w * a.G) - 1;
  const int p0 = r.L - r.w;
  TileRange t;
  t.lo = a.window ? window_low(a, p0 + row0 / a.G) & ~15 : 0;
  t.hi = a.causal ? causal_high(a, r, p0 + row1 / a.G) : r.L;
  t.steps = t.hi > t.lo ? (t.hi - t.lo + kTileKeys - 1) / kTileKeys : 1;
  return t;
}

// Beginning and ending an item (queries, result) costs a block about as much as this
// many steps; shares count an item as kItemCost + steps.  (The chunks and the candidates
// named below: 1 gives 247 and 258 us, 2 226 and 255, 3 228 and 270, 4 232 and 281.)
constexpr int kItemCost = 2;

// Walks the items (request, kv head, row tile) of a block's share of the work, the
// same way in every warp.  A share that holds only the first kItemCost units of an
// item leaves it to the next one.
struct TileWalk {
  long long u, u_end;
  Request req;
  long long head_units;  // cost of one head of the request
  TileRange range;
  int tiles, tile, b, h, x0, x1;  // the share takes units [x0, x1) of the item,
  int s0, s1;                     // which are its steps [s0, s1)

  __device__ __forceinline__ static long long cost_of(const AttendArgs& a, const Request& r,
                                                       int from, int stride) {
    long long x = 0;
    const int n = (r.w * a.G + kTileRows - 1) / kTileRows;
    if (!a.causal && !a.window)  // every tile sees every key
      return from < n ? ((n - 1 - from) / stride + 1ll) * (kItemCost + tile_range(a, r, 0).steps) : 0;
    for (int t = from; t < n; t += stride) x += kItemCost + tile_range(a, r, t).steps;
    return x;
  }
  // Whole-warp: the cost of one head of the request.
  __device__ __forceinline__ void enter(const AttendArgs& a, int to) {
    b = to;
    req = request_of(a, b, false);
    tiles = (req.w * a.G + kTileRows - 1) / kTileRows;
    long long x = cost_of(a, req, threadIdx.x & 31, 32);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
    head_units = x;
  }
  // The share [first, end) begins `into` steps into request b.
  __device__ __forceinline__ void start(const AttendArgs& a, int at, long long into, long long first,
                                        long long end) {
    u = first;
    u_end = end;
    enter(a, at);
    h = (int)(into / head_units);
    into -= h * head_units;
    tile = 0;
    range = tile_range(a, req, 0);
    while (into >= kItemCost + range.steps) {
      into -= kItemCost + range.steps;
      range = tile_range(a, req, ++tile);
    }
    x0 = (int)into;
    cut();
    if (s0 == s1) next(a);
  }
  __device__ __forceinline__ void cut() {
    x1 = (int)min((long long)(kItemCost + range.steps), x0 + (u_end - u));
    s0 = max(0, x0 - kItemCost);
    s1 = max(0, x1 - kItemCost);
  }
  // To the next item with steps in the share; s0 == s1 and false where there is none.
  __device__ __forceinline__ bool next(const AttendArgs& a) {
    u += x1 - x0;
    if (u >= u_end) {
      s0 = s1 = 0;
      return false;
    }
    if (++tile == tiles) {
      tile = 0;
      if (++h == a.H) {
        h = 0;
        do enter(a, b + 1);
        while (tiles == 0);
      }
    }
    range = tile_range(a, req, tile);
    x0 = 0;
    cut();
    return s1 > s0;  // a share that ends inside the cost of an item has nothing behind it
  }
  __device__ __forceinline__ bool begins() const { return s0 == 0; }
  __device__ __forceinline__ bool ends() const { return s1 == range.steps; }
  // Block whose share ends the item.
  __device__ __forceinline__ int last_block(long long per) const {
    return (int)((u - x0 + kItemCost + range.steps - 1) / per);
  }
};

// What the other warps need of an item; steps == 0 ends the list.
struct TileItem {
  int b, h, tile, start, w, L;
  int key0;            // first key of the share's steps
  int steps;
  int whole;           // bit 0: the share holds the item's first step, bit 1: its last
  int last;            // block whose share ends the item
};

struct TileSmall {
  uint64_t full[2][kTileStages], free[2][kTileStages];  // [K, V]
  uint64_t raw_full[kRawSlots], raw_free[kRawSlots];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], scales[kScaleSlots];
  uint64_t item_full[kItems], item_free[kItems];
  float2 scale[kScaleSlots][kGroups];  // |key scale|, log2 |value scale| of a group
  float top[kScaleSlots];              // largest finite |value scale| of the step
  uint32_t hidden[kScaleSlots];        // bit g: group g has no block
  uint32_t negative[kScaleSlots];      // bit g, 8 + g: its key, value scale is negative
  TileItem items[kItems];
  int32_t failed;
  uint32_t tmem;
  int32_t b;
  int32_t pad;
  long long before;
  long long sums[kTileThreads / 32];
  // [half][columns][row], read by the row's other thread; maxima are written again only
  // behind the next step's barrier, sums behind the next item's
  float2 swap_max[2][2][128];  // and the largest p * value scale over it, log2
  float swap_sum[2][2][128];
};
static_assert(sizeof(TileSmall) <= 8192);

__device__ __forceinline__ bool any_of_256(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\n"
      "barrier.cta.red.or.pred q, %1, 256, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_256(int id) {
  asm volatile("barrier.cta.sync %0, 256;" ::"r"(id) : "memory");
}
// 8 words of one 32-byte sector.
__device__ __forceinline__ void store32(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
               "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// 8 codes (two words) as 16 bytes of bf16, times sign (+-1): 0x4300 | low 7 bits is
// 128 + low, 0x4300 | bit 7 is 128 or 256, and their difference is the code, exactly.
__device__ __forceinline__ uint4 codes_to_bf8(uint2 w, bool minus) {
  uint32_t h[4];
  const uint32_t sign2 = minus ? 0xBF80BF80u : 0x3F803F80u, flip = minus ? 0u : 0x80008000u;
  const uint32_t m[4] = {__byte_perm(w.x, 0x43434343u, kSelLow), __byte_perm(w.x, 0x43434343u, kSelHigh),
                         __byte_perm(w.y, 0x43434343u, kSelLow), __byte_perm(w.y, 0x43434343u, kSelHigh)};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(h[i])
        : "r"(m[i] & 0xFF7FFF7Fu), "r"(sign2), "r"((m[i] & 0xFF80FF80u) ^ flip));
  return make_uint4(h[0], h[1], h[2], h[3]);
}
// 8 codes (two words) as 16 bytes of fp16, times sign (+-1).
__device__ __forceinline__ uint4 codes_to_half8(uint2 w, uint32_t sign2, uint32_t off2) {
  uint32_t h[4];
  const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
  const uint32_t m[4] = {__byte_perm(x, 0x64646464u, kSelLow), __byte_perm(x, 0x64646464u, kSelHigh),
                         __byte_perm(y, 0x64646464u, kSelLow), __byte_perm(y, 0x64646464u, kSelHigh)};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h[i]) : "r"(m[i]), "r"(sign2), "r"(off2));
  return make_uint4(h[0], h[1], h[2], h[3]);
}
__device__ __forceinline__ void sts16(uint32_t to, uint4 y) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
               : "memory");
}
constexpr uint32_t kPlus2 = 0x3C003C00u, kMinus2 = 0xBC00BC00u;      // 1, -1
constexpr uint32_t kOffPlus2 = 0xE480E480u, kOffMinus2 = 0x64806480u;  // -1152, 1152

// One block an SM.  Per step of 128 keys a loader warp brings the codes of K and V into
// shared memory (bulk copies of 16 tokens, three slots of 64), a converter warpgroup
// turns them into 16-bit operands there (two stages), one thread issues
//   S_i = Q_i K^T (i = 0, 1: the two halves of 128 rows), O_i += P_i V
// with S and O in TMEM, and two warpgroups for each half turn S_i into P_i, a thread
// taking 64 of a row's 128 keys.  P_i takes the place of S_i in TMEM as fp16 pairs.  The
// halves alternate (P_0 V, Q_0 K', P_1 V, Q_1 K'), so that one half's exponentials run
// under the other's products.  What bounds it is the chain of one half: per step about
// 3,600 cycles of softmax (of which the exponentials, 4 lanes a cycle and scheduler
// shared by four warps, take 1,550), then 1,300 of its two products and 600 of signals,
// of 6,000 in all; the tensor pipe is busy 0.30 of the time.  Six chunks of 500 to 4,096
// rows behind up to 8,000 keys, 16 query and 4 kv heads x 128, bf16 (133 GFLOP): 226 us,
// 590 TFLOP/s, 0.36 of the measured matrix rate; 32 x 1,024 candidates, 8 heads x 64, fp16
// (72 GFLOP): 255 us (222 before the weights' second part).  What it went through: one thread a row with 128 keys 660 us; bulk
// copies and smaller code (the roles together overran the instruction cache) 513;
// queries copied under the last step 373; two threads a row 283; item cost in the shares
// 250; products issued from warp-uniform code 233.  Scales: the score factor holds the key scale (one for 16
// keys); the value scale goes into the exponent, p 2^7 scale / 2^ev =
// 2^(s - m + log2(scale) + 7 - ev), and the row sum takes it out again once in 16 keys, so
// neither costs work per element.  O is rescaled only when a row's maximum or its largest
// product p * scale, which ev follows, rises by more than 2^kSlack.
// The loader warp also walks the block's items and hands them to the others.  A wait
// that runs out marks the launch failed and lets every role run to its end without
// further waits, so that all named barriers are met.
template <int D, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) k_kv_tiles(AttendArgs a) {
  pdl_enter();
  pdl_trigger();
  using L = TileSmem<D>;
  constexpr bool kBf16 = __is_same(T, __nv_bfloat16);  // queries and keys go as they are
  // fp16 results get the weights in two fp16 parts: with one they were 1.4 to 1.5 times as
  // far from 64 bits as their own rounding (3.0e-4 against 2.1e-4); bf16's hides it.
  constexpr bool kTwo = !kBf16;
  extern __shared__ __align__(16) uint8_t s_tile[];
  const uint32_t base = (smem_addr(s_tile) + 1023) & ~1023u;
  TileSmall* sm = reinterpret_cast<TileSmall*>(s_tile + (base - smem_addr(s_tile)) + L::kSmall);
  // through a shuffle, so that the compiler knows it to be the same in all lanes
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  constexpr int kWarps = kTileThreads / 32;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sm->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < kTileStages; ++i) {
        bar_init(&sm->full[w][i], 32 * kConvWarps);
        bar_init(&sm->free[w][i], 1);
      }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm->q_full[i], 256);
      bar_init(&sm->p_full[i], 256);
      bar_init(&sm->s_full[i], 1);
      bar_init(&sm->o_full[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) bar_init(&sm->scales[i], 1);
    for (int i = 0; i < kRawSlots; ++i) {
      bar_init(&sm->raw_full[i], 1);
      bar_init(&sm->raw_free[i], 32 * kConvWarps);
    }
    for (int i = 0; i < kItems; ++i) {
      bar_init(&sm->item_full[i], 1);
      bar_init(&sm->item_free[i], kSoftWarps + kConvWarps + 1);
    }
    sm->failed = 0;
    sm->b = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();

  // ---- this block's share: a warp's lanes take a request's tiles where requests are
  // few, a thread a request where they are many; chunks in request order
  const bool by_warp = a.B < kTileThreads;
  const int workers = by_warp ? kWarps : kTileThreads, me = by_warp ? warp : tid;
  const int per_worker = (a.B + workers - 1) / workers;
  const int b_lo = min(a.B, me * per_worker), b_hi = min(a.B, b_lo + per_worker);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Request r = request_of(a, b, blockIdx.x == 0);
    mine += TileWalk::cost_of(a, r, by_warp ? lane : 0, by_warp ? 32 : 1) * a.H;
  }
  long long incl = mine;  // inclusive over lanes
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sm->sums[warp] = incl;
  __syncthreads();
  tc_fence_after();
  long long total = 0, before = 0;
#pragma unroll 1
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sm->sums[i];
    total += sm->sums[i];
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < 1) per = 1;
  const long long u0 = per * blockIdx.x, u_end = min(total, u0 + per);
  {
    // the worker whose requests hold unit u0 walks them
    const long long from = by_warp ? before : before + incl - mine;
    const long long to = by_warp ? before + sm->sums[warp] : before + incl;
    if (from <= u0 && u0 < to) {
      long long at = from;
      for (int b = b_lo; b < b_hi; ++b) {
        const Request r = request_of(a, b, false);
        long long x = TileWalk::cost_of(a, r, by_warp ? lane : 0, by_warp ? 32 : 1) * a.H;
        if (by_warp) {
#pragma unroll
          for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
        }
        if (at + x > u0) {
          if (!by_warp || lane == 0) {
            sm->b = b;
            sm->before = at;
          }
          break;
        }
        at += x;
      }
    }
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(kAll, sm->tmem, 0);
  volatile int32_t* failed = &sm->failed;

  // Item i; false where the wait ran out.
  auto item_wait = [&](uint32_t i) {
    return bar_wait(&sm->item_full[i % kItems], (i / kItems) & 1, failed, a.status);
  };
  auto item_done = [&](uint32_t i) {  // the warp has read it
    __syncwarp();
    if (lane == 0) bar_arrive(&sm->item_free[i % kItems]);
  };

  if (warp < kSoftWarps) {
    // ================================================================ softmax
    const int half = warp >> 3, part = warp >> 2 & 1;
    const int at_row = (warp & 3) * 32 + lane;  // of the half = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + half * 128 + part * 64 + lanes;           // 64 scores
    const uint32_t t_o = tmem + 256 + half * D + part * (D / 2) + lanes;  // D / 2 outputs
    const float inv = fabsf(a.scale_log2);
    // The row's queries go into shared memory as they are (products of 16-bit values
    // with codes are exact), 16 bytes a copy, half of them by each thread of the row.
    // The next item's are asked for when the last scores of this one are there, and so
    // come under its last step.
    auto fetch_q = [&](const TileItem& w) {
      const int row = w.tile * kTileRows + half * 128 + at_row;
      const bool real = row < w.w * a.G;
      const int t = real ? row / a.G : 0;
      const T* q = static_cast<const T*>(a.q) + (w.start + t) * a.qsn +
                   (w.h * a.G + (real ? row - t * a.G : 0)) * a.qsh + part * (D / 2);
      const uint32_t q_at = base + L::kQ + half * L::kOperand + at_row * 128 +
                            (D == 128 ? part * L::kPlane : 0);
#pragma unroll
      for (int d = 0; d < D / 2; d += 8) {
        const uint32_t to = q_at + ((((D == 128 ? 0 : part * 32) + d) * 2) ^ ((at_row & 7) << 4));
        if (real)
          copy16(to, reinterpret_cast<const int8_t*>(q + d));
        else
          sts16(to, make_uint4(0, 0, 0, 0));
      }
      copies_commit();
    };
    auto has_rows = [&](const TileItem& w) {
      return w.steps > 0 && w.tile * kTileRows + half * 128 < w.w * a.G;
    };
    auto publish_q = [&] {
      copies_wait<0>();
      proxy_fence();
      bar_arrive(&sm->q_full[half]);
    };
    uint32_t n_s = 0, n_o = 0, n_k = 0;  // s_full and o_full phases, steps so far
    PartHead head = {0, 0, 0, -1};
    bool asked = false;  // this item's queries are on their way
    for (uint32_t it = 0;; ++it) {
      // the 256 threads of a half agree on going on
      if (any_of_256(1 + half, !item_wait(it))) break;
      const TileItem item = sm->items[it % kItems];
      if (item.steps == 0) break;
      if (!asked && has_rows(item)) {
        fetch_q(item);
        publish_q();
      }
      item_done(it);
      const bool begins = item.whole & 1, whole = item.whole == 3;
      if (begins && !whole) {
        head.b = item.b;
        head.h = item.h;
        head.tile = item.tile;
        head.last = item.last;
      }
      const bool here = has_rows(item);
      asked = false;
      const int row = item.tile * kTileRows + half * 128 + at_row;
      const bool real = row < item.w * a.G;
      const int t = real ? row / a.G : 0;
      const int pos = item.L - item.w + t;
      const int hi = real ? (a.causal ? max(0, min(item.L, pos + 1)) : item.L) : 0;
      const int lo = window_low(a, pos);
      if (!here) {  // this half of the tile is empty
        n_k += item.steps;
        continue;
      }
      float m = -CUDART_INF_F, sum = 0.f;
      bool seen = false;             // a key of this share
      float d = -CUDART_INF_F, ev = 0.f;  // log2 of the largest p * value scale, reference
      float vtop = 0.f, least = kLeastRef;
#pragma unroll 1
      for (int j = 0; j < item.steps; ++j, ++n_k) {
        const int key = item.key0 + j * kTileKeys + part * 64;
        const int slot = n_k % kScaleSlots;
        bar_wait(&sm->scales[slot], (n_k / kScaleSlots) & 1, failed, a.status);
        bar_wait(&sm->s_full[half], n_s & 1, failed, a.status);
        ++n_s;
        __syncwarp();
        tc_fence_after();
        if (j == item.steps - 1) {
          if (item_wait(it + 1) && has_rows(sm->items[(it + 1) % kItems])) {
            fetch_q(sm->items[(it + 1) % kItems]);
            asked = true;
          }
          __syncwarp();
        }
        const float2* scale = &sm->scale[slot][part * 4];
        const float va = sm->top[slot];
        const uint32_t none = sm->hidden[slot] >> part * 4 & 0xF;
        // does every row of the warp see every key?  (real rows; the others' results
        // are not used)
        const bool hide = none || __any_sync(kAll, real && (key + 64 > hi || key < lo));
        // keys that this row sees: in [lo, hi) and of a block that is there
        auto visible = [&](int cnk) {
          const uint32_t gone = none >> (cnk * 2);
          return keys_between(key + cnk * 32, lo, hi) & ((gone & 1 ? 0 : 0xFFFFu) |
                                                        (gone & 2 ? 0 : 0xFFFF0000u));
        };
        // ---- largest score.  The loops over 32 keys stay loops: unrolled, the block's
        // roles together overran the instruction cache.
        float mx = -CUDART_INF_F, mv = -CUDART_INF_F;  // (mv: over 2^mx)
#pragma unroll 1
        for (int cnk = 0; cnk < 2; ++cnk) {
          uint32_t y[32];
          tmem_load32(t_s + cnk * 32, y);
          tmem_loaded(y);
          if (hide) {
            const uint32_t vis = visible(cnk);
            seen |= vis != 0;
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = vis >> e & 1 ? y[e] : 0xFF800000u;
          }
          float top[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float f = __fmul_rn(inv, scale[cnk * 2 + g].x);
            const float* z = reinterpret_cast<const float*>(y) + g * 16;
            float best = max3(max3(z[0], z[1], z[2]), max3(z[3], z[4], z[5]), max3(z[6], z[7], z[8]));
            best = max3(best, max3(z[9], z[10], z[11]), max3(z[12], z[13], z[14]));
            best = fmaxf(best, z[15]);
            top[g] = best > -CUDART_INF_F ? __fmul_rn(best, f) : -CUDART_INF_F;
          }
          const float to = max3(mx, top[0], top[1]);
          mv = max3(mv + (mx - to), top[0] - to + scale[cnk * 2].y, top[1] - to + scale[cnk * 2 + 1].y);
          mx = to;
        }
        seen |= !hide;
        const bool vup = va > vtop;
        if (any_of_256(1 + half, mx > m + kSlack || mx - m + mv > d + kSlack || vup)) {
          sm->swap_max[half][part][at_row] = make_float2(mx, mv);
          sync_256(1 + half);
          const float2 other = sm->swap_max[half][part ^ 1][at_row];
          const float both = fmaxf(mx, other.x);
          mv = fmaxf(mv + (mx - both), other.y + (other.x - both));  // (NaN: no key)
          if (vup) raise_top(va, vtop, least);
          const float to = fmaxf(m, both);
          const float alpha = to == m ? 1.f : exp2_fast(m - to);
          if (to != m) d += m - to;
          d = fmaxf(d, mv + (both - to));
          const float ev0 = ev;
          ev = row_ref(d, least);
          m = to;
          sum = __fmul_rn(sum, alpha);
          if (j > 0) {
            const float g = __fmul_rn(alpha, exp2_whole(fminf(fmaxf(ev0 - ev, -126.f), 127.f)));
#pragma unroll 1
            for (int d = 0; d < D / 2; d += 32) {
              uint32_t x[32];
              tmem_load32(t_o + d, x);
              tmem_loaded(x);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__fmul_rn(__uint_as_float(x[e]), g));
              tmem_store32(t_o + d, x);
            }
            tmem_stored();
          }
        }
        // ---- weights.  Scores beyond 2^20 in log2 units are rounded like the maximum
        // before it is taken off; below, one fma does.
        const float top = m == -CUDART_INF_F ? 0.f : m;
        const bool big = __any_sync(kAll, fabsf(top) > 1048576.f);
        uint32_t low[16];  // kTwo: second parts, which wait until their place has been read
#pragma unroll 1
        for (int cnk = 0; cnk < 2; ++cnk) {
          uint32_t y[32];
          tmem_load32(t_s + cnk * 32, y);
          float* p = reinterpret_cast<float*>(y);
          float lp[2], f[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 sc = scale[cnk * 2 + g];
            f[g] = __fmul_rn(inv, sc.x);
            // log2 of 2^7 scale / 2^ev; far below, the weights vanish in fp16 anyway
            const float x = __fadd_rn(__fsub_rn(sc.y, ev), 7.f);
            lp[g] = x < -60.f ? -60.f : x;
          }
          tmem_loaded(y);
          if (kTwo && cnk == 1) tmem_store16(t_s + 32, low);
          if (big) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              p[e] = __fadd_rn(__fsub_rn(__fmul_rn(p[e], f[e >> 4]), top), lp[e >> 4]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float off = __fsub_rn(lp[e >> 4], top);
              unpair(fma2(pair(p[e], p[e + 1]), pair(f[e >> 4], f[e >> 4]), pair(off, off)), p[e],
                     p[e + 1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) p[e] = exp2_fast(p[e]);
          if (hide) {
            const uint32_t vis = visible(cnk);
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = vis >> e & 1 ? p[e] : 0.f;
          }
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint64_t s2[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s2[e] = add2(pair(p[g * 16 + 4 * e], p[g * 16 + 4 * e + 1]),
                           pair(p[g * 16 + 4 * e + 2], p[g * 16 + 4 * e + 3]));
            float s0, s1;
            unpair(add2(add2(s2[0], s2[1]), add2(s2[2], s2[3])), s0, s1);
            s0 = __fadd_rn(s0, s1);
            if (s0 != 0.f) sum = __fmaf_rn(s0, exp2_fast(-lp[g]), sum);
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            pk[e] = half2_bits(p[2 * e], p[2 * e + 1]);
            if constexpr (kTwo) {
              const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&pk[e]));
              low[e] = half2_bits(__fsub_rn(p[2 * e], h.x), __fsub_rn(p[2 * e + 1], h.y));
            }
          }
          tmem_store16(t_s + cnk * 16, pk);
        }
        if (kTwo) tmem_store16(t_s + 48, low);
        tmem_stored();
        tc_fence_before();
        bar_arrive(&sm->p_full[half]);
      }
      if (asked) publish_q();
      // ---- the row's result: the partner's sum, then D / 2 outputs each
      // (-0: nothing but weights of 0, from keys that were seen)
      sm->swap_sum[half][part][at_row] = seen && sum == 0.f ? -0.f : sum;
      sync_256(1 + half);
      const float other = sm->swap_sum[half][part ^ 1][at_row];
      seen |= __float_as_uint(other) == 0x80000000u;
      sum = __fadd_rn(fabsf(other), sum);
      // the largest score has weight 1 at least, so every score was -inf: a query that is
      // not finite
      if (seen && sum == 0.f) sum = CUDART_NAN_F;
      bar_wait(&sm->o_full[half], n_o & 1, failed, a.status);
      ++n_o;
      __syncwarp();
      tc_fence_after();
      const int hq = item.h * a.G + (real ? row - t * a.G : 0);
      const float unit = exp2_whole(ev - 7.f);
      // the mean, also of a part, in two steps, since unit / sum can underflow
      const float g = __fdiv_rn(1.f, sum);
      const int prow = half * 128 + at_row;
      float* out_part = a.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kTileRows * (D + 2) +
                        prow * D + part * (D / 2);
      T* out = static_cast<T*>(a.out) + (item.start + t) * a.osn + hq * a.osh + part * (D / 2);
#pragma unroll 1
      for (int d = 0; d < D / 2; d += 32) {
        uint32_t x[32];
        tmem_load32(t_o + d, x);
        tmem_loaded(x);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          // a row that saw no key: 0, whatever the hidden blocks hold
          x[e] = sum == 0.f ? 0u : __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(x[e]), g), unit));
        if (!real) continue;
        if (whole) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float lo2 = __uint_as_float(x[2 * e]), hi2 = __uint_as_float(x[2 * e + 1]);
            if constexpr (kBf16) {
              const __nv_bfloat162 h2 = __floats2bfloat162_rn(lo2, hi2);
              y[e] = *reinterpret_cast<const uint32_t*>(&h2);
            } else {
              y[e] = half2_bits(lo2, hi2);
            }
          }
          if (a.out_sectors) {
            store32(out + d, y);
            store32(out + d + 16, y + 8);
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(out + d + 2 * e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) store32(out_part + d + e, x + e);
        }
      }
      if (real && part == 0) {
        if (!whole)
          *reinterpret_cast<float2*>(out_part - prow * D + kTileRows * D + prow * 2) =
              make_float2(m, sum);
        else if (a.lse)
          a.lse[(int64_t)(item.start + t) * a.Hq + hq] =
              sum == 0.f ? -CUDART_INF_F : __fmul_rn(m + log2f(sum), 0.6931471805599453f);
      }
      tc_fence_before();
    }
    if (tid == 0) a.heads[blockIdx.x] = head;
  } else if (warp < kMmaWarp) {
    // ================================================================ converters
    // A thread takes 16 codes of a key at a time; the lanes of the upper plane store
    // their two halves in the other order, so that a phase of 8 lanes hits all banks.
    const int ct = tid - 32 * kSoftWarps;
    constexpr int kCols = D / 16, kKeys = 32 * kConvWarps / kCols;  // keys of a round
    const int col = ct % kCols, key_in = ct / kCols;
    const bool swap = col >= 4;
    uint32_t n_k = 0, n_raw = 0;
    for (uint32_t it = 0;; ++it) {
      if (!__all_sync(kAll, item_wait(it))) break;
      const int n_steps = sm->items[it % kItems].steps;
      item_done(it);
      if (n_steps == 0) break;
#pragma unroll 1
      for (int piece = 0; piece < 4 * n_steps; ++piece, ++n_raw) {
        const int which = piece >> 1 & 1, low = piece & 1, stage = n_k % kTileStages;
        const int slot = n_raw % kRawSlots;
        if (low == 0)
          bar_wait(&sm->free[which][stage], ((n_k / kTileStages) & 1) ^ 1, failed, a.status);
        bar_wait(&sm->raw_full[slot], (n_raw / kRawSlots) & 1, failed, a.status);
        const uint32_t from = base + L::kRaw + slot * (kRawKeys * D) + ct * 16;
        const uint32_t to = base + (which ? L::kV : L::kK) + stage * L::kOperand + low * (kRawKeys * 128) +
                            (col / 4) * L::kPlane;
        // a negative scale (no append gives one) goes into the codes' sign
        const uint32_t neg = sm->negative[n_k % kScaleSlots] >> (which * kGroups + low * 4);
        uint32_t w[kRawKeys / kKeys][4];
#pragma unroll
        for (int i = 0; i < kRawKeys / kKeys; ++i) lds_words<4>(from + i * (kKeys * D), w[i]);
#pragma unroll
        for (int i = 0; i < kRawKeys / kKeys; ++i) {
          const int row = i * kKeys + key_in;
          const bool minus = neg >> (row >> 4) & 1;
          const uint2 lo2 = swap ? make_uint2(w[i][2], w[i][3]) : make_uint2(w[i][0], w[i][1]);
          const uint2 hi2 = swap ? make_uint2(w[i][0], w[i][1]) : make_uint2(w[i][2], w[i][3]);
          const uint32_t at = to + row * 128;
          const uint32_t x = (col % 4) * 32 + (swap ? 16 : 0);
          uint4 y0, y1;
          if (kBf16 && which == 0) {
            y0 = codes_to_bf8(lo2, minus);
            y1 = codes_to_bf8(hi2, minus);
          } else {
            const uint32_t sign2 = minus ? kMinus2 : kPlus2, off2 = minus ? kOffMinus2 : kOffPlus2;
            y0 = codes_to_half8(lo2, sign2, off2);
            y1 = codes_to_half8(hi2, sign2, off2);
          }
          sts16(at + (x ^ ((row & 7) << 4)), y0);
          sts16(at + ((x ^ 16) ^ ((row & 7) << 4)), y1);
        }
        bar_arrive(&sm->raw_free[slot]);
        if (low) {
          proxy_fence();
          bar_arrive(&sm->full[which][stage]);
          if (which) ++n_k;
        }
      }
    }
  } else if (warp == kLoadWarp) {
    // ================================================================ loader
    TileWalk walk;
    uint32_t n_items = 0;
    bool more = u0 < u_end;
    if (more) {
      walk.start(a, sm->b, u0 - sm->before, u0, u_end);
      more = walk.s1 > walk.s0;
    }
    auto publish = [&] {  // the walk's item, or the end of the list
      const int slot = n_items % kItems;
      bar_wait(&sm->item_free[slot], ((n_items / kItems) & 1) ^ 1, failed, a.status);
      if (lane == 0) {
        TileItem* x = &sm->items[slot];
        x->steps = more ? walk.s1 - walk.s0 : 0;
        if (more) {
          x->b = walk.b;
          x->h = walk.h;
          x->tile = walk.tile;
          x->start = walk.req.start;
          x->w = walk.req.w;
          x->L = walk.req.L;
          x->key0 = walk.range.lo + walk.s0 * kTileKeys;
          x->whole = (walk.begins() ? 1 : 0) | (walk.ends() ? 2 : 0);
          x->last = walk.last_block(per);
        }
        bar_arrive(&sm->item_full[slot]);
      }
      __syncwarp();
      ++n_items;
    };
    // Lane g < 8 has 16-key group g of a step: its block id (-1: none, its keys are
    // hidden), scales, and the copies of its 16 x D codes of K and of V.
    const int bs = 1 << a.bs_log;
    const int64_t block_bytes = ((int64_t)a.H << a.bs_log) * D;
    uint32_t n_k = 0, n_raw = 0;
    publish();
    for (uint32_t it = 0; more; ++it) {
      const int b = walk.b, h = walk.h, n_steps = walk.s1 - walk.s0, hi = walk.range.hi;
      const int key0 = walk.range.lo + walk.s0 * kTileKeys + lane * 16;
      more = walk.next(a);
      publish();  // the next one, while this one's codes are brought
      const int32_t* row_table = a.table + (int64_t)b * a.max_blocks;
      const int64_t head_at = ((int64_t)h << a.bs_log) * D;
      auto look_up = [&](int j, int32_t& id, float& ks, float& vs) {
        id = -1;
        ks = vs = 0.f;
        const int key = key0 + j * kTileKeys;
        if (lane < kGroups && j < n_steps && key < hi) {
          id = __ldg(row_table + (key >> a.bs_log));
          if (id < 0 || id >= a.num_blocks) {
            id = -1;
            set_status(a.status, kStBadBlock);
          } else {
            ks = __ldg(a.ks + (int64_t)id * a.H + h);
            vs = __ldg(a.vs + (int64_t)id * a.H + h);
          }
        }
      };
      int32_t id, id_n;
      float ks, vs, ks_n, vs_n;
      look_up(0, id, ks, vs);
#pragma unroll 1
      for (int j = 0; j < n_steps; ++j, ++n_k) {
        look_up(j + 1, id_n, ks_n, vs_n);
        const uint32_t there = __ballot_sync(kAll, id >= 0);
        const int64_t off = id * block_bytes + head_at + ((key0 + j * kTileKeys) & (bs - 1)) * D;
#pragma unroll 1
        for (int q = 0; q < 4; ++q, ++n_raw) {
          const int slot = n_raw % kRawSlots;
          bar_wait(&sm->raw_free[slot], ((n_raw / kRawSlots) & 1) ^ 1, failed, a.status);
          __syncwarp();
          if (q == 0) {
            // every reader of this slot's last step is behind: keys of the step before
            // this one have been converted, so the products of the step before that
            // were issued, and so the weights of the step before those were ready
            const int sl = n_k % kScaleSlots;
            const uint32_t nk = __ballot_sync(kAll, ks < 0.f), nv = __ballot_sync(kAll, vs < 0.f);
            if (lane < kGroups) sm->scale[sl][lane] = make_float2(fabsf(ks), log2f(fabsf(vs)));
            float top = lane < kGroups && fabsf(vs) < CUDART_INF_F ? fabsf(vs) : 0.f;
            top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(top)));
            if (lane == 0) {
              sm->top[sl] = top;
              sm->hidden[sl] = ~there & ((1u << kGroups) - 1);
              // a negative softmax scale turns the keys' sign too
              sm->negative[sl] = (a.scale_log2 < 0.f ? ~nk & 0xFF : nk) | nv << kGroups;
            }
            __syncwarp();
            if (lane == 0) bar_arrive(&sm->scales[sl]);
          }
          const uint32_t mine4 = there >> (q & 1) * 4 & 0xF;
          if (lane == 0) bar_expect(&sm->raw_full[slot], __popc(mine4) * (16 * D));
          __syncwarp();
          if (id >= 0 && (lane >> 2) == (q & 1))
            copy_bulk(base + L::kRaw + slot * (kRawKeys * D) + (lane & 3) * (16 * D),
                      (q < 2 ? a.k : a.v) + off, 16 * D, &sm->raw_full[slot]);
        }
        id = id_n;
        ks = ks_n;
        vs = vs_n;
      }
    }
    // the last copies have landed (again with a limit) before the block may end
    for (uint32_t i = n_raw < kRawSlots ? 0 : n_raw - kRawSlots; i < n_raw; ++i) {
      const uint64_t t0 = global_ns();
      while (!bar_test(&sm->raw_full[i % kRawSlots], (i / kRawSlots) & 1) &&
             global_ns() - t0 < kWaitLimitNs) {
      }
    }
  } else {
    // ================================================================ products
    uint32_t n_k = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};
    const uint32_t leader = lane == 0;
    constexpr uint32_t kScores = instruction<kTileKeys, false, kBf16>();
    constexpr uint32_t kOut = instruction<D, true, false>();
    constexpr uint32_t kHigh = operand_high(1024);
    for (uint32_t it = 0;; ++it) {
      if (!__all_sync(kAll, item_wait(it))) break;
      const int n_steps = __shfl_sync(kAll, sm->items[it % kItems].steps, 0);
      const int rows = __shfl_sync(
          kAll, sm->items[it % kItems].w * a.G - sm->items[it % kItems].tile * kTileRows, 0);
      item_done(it);
      if (n_steps == 0) break;
      const int halves = rows > 128 ? 2 : 1;
      {
        auto scores = [&](int i, uint32_t step) {
          const uint32_t q = operand_low(base + L::kQ + i * L::kOperand, 16);
          const uint32_t k = operand_low(base + L::kK + (step % kTileStages) * L::kOperand, 16);
          const uint32_t d = tmem + i * 128;
#pragma unroll
          for (int pl = 0; pl < D / 64; ++pl)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t at = (pl * L::kPlane + kk * 32) >> 4;
              mma_ss(leader, d, q + at, k + at, kHigh, kScores, (pl | kk) != 0);
            }
          tc_commit(leader, &sm->s_full[i]);
        };
        for (int i = 0; i < halves; ++i) bar_wait(&sm->q_full[i], n_q[i]++ & 1, failed, a.status);
        bar_wait(&sm->full[0][n_k % kTileStages], (n_k / kTileStages) & 1, failed, a.status);
        tc_fence_after();
        for (int i = 0; i < halves; ++i) scores(i, n_k);
        tc_commit(leader, &sm->free[0][n_k % kTileStages]);
#pragma unroll 1
        for (int j = 0; j < n_steps; ++j, ++n_k) {
          const int stage = n_k % kTileStages;
          bar_wait(&sm->full[1][stage], (n_k / kTileStages) & 1, failed, a.status);
#pragma unroll 1
          for (int i = 0; i < halves; ++i) {
            bar_wait(&sm->p_full[i], n_p[i]++ & 1, failed, a.status);
            tc_fence_after();
            const uint32_t v = operand_low(base + L::kV + stage * L::kOperand, L::kPlane);
            const uint32_t d = tmem + 256 + i * D, p = tmem + i * 128;
#pragma unroll
            for (int kk = 0; kk < kTileKeys / 16; ++kk)
              mma_ts(leader, d, p + (kk / 4) * 64 + (kk % 4) * 8, v + kk * (2048 >> 4), kHigh, kOut,
                     kk > 0 || j > 0);
            if constexpr (kTwo) {
#pragma unroll
              for (int kk = 0; kk < kTileKeys / 16; ++kk)
                mma_ts(leader, d, p + (kk / 4) * 64 + 32 + (kk % 4) * 8, v + kk * (2048 >> 4), kHigh,
                       kOut, true);
            }
            if (i == halves - 1) tc_commit(leader, &sm->free[1][stage]);
            if (j == n_steps - 1) {
              tc_commit(leader, &sm->o_full[i]);
            } else {
              if (i == 0) {
                const uint32_t nx = n_k + 1;
                bar_wait(&sm->full[0][nx % kTileStages], (nx / kTileStages) & 1, failed, a.status);
                tc_fence_after();
              }
              scores(i, n_k + 1);
              if (i == halves - 1) tc_commit(leader, &sm->free[0][(n_k + 1) % kTileStages]);
            }
          }
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace mpzch_kv
