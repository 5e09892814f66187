// Attention over the history cache for many rows per request (admissions, chunks,
// candidates): 256-row tiles on the tensor cores (tcgen05, accumulators in TMEM).
#pragma once
#include "mpzch_kv_rows.cuh"

namespace mpzch_kv {

constexpr int kTileRows = 256;   // two halves of 128, each with its softmax warpgroup
constexpr int kTileKeys = 128;   // keys of one step
constexpr int kGroups = kTileKeys / 16;
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kTileThreads = 32 * (kSoftWarps + kConvWarps + 1);
constexpr int kTileStages = 2;
constexpr int kScaleSlots = 4;

// Shared memory: Q [2 halves][D / 64][128 rows][128 B], K and V stages
// [D / 64][128 keys][128 B], all in the 128-byte swizzle, then the small fields.
template <int D>
struct TileSmem {
  static constexpr int kPlane = 128 * 128;            // 64 dims of 128 rows
  static constexpr int kOperand = D / 64 * kPlane;
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kOperand;
  static constexpr int kV = kK + kTileStages * kOperand;
  static constexpr int kSmall = kV + kTileStages * kOperand;
  static constexpr int kBytes = kSmall + 1024 + 1024;  // and up to 1 KB to align the base
};

struct TileSmall {
  uint64_t k_full[kTileStages], v_full[kTileStages], k_free[kTileStages], v_free[kTileStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], scales[kScaleSlots];
  float ks[kScaleSlots][kGroups], vs[kScaleSlots][kGroups];
  uint32_t hidden[kScaleSlots];  // bit g: group g has no block
  uint32_t tmem;
  int32_t failed;
  int32_t b;
  int32_t pad;
  long long units, before;
  long long sums[16];
};
static_assert(sizeof(TileSmall) <= 1024);

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
// Waits for a phase; gives up after kWaitLimitNs (then, and once any warp of the
// block gave up, false).
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, TileSmall* sm,
                                         int32_t* status) {
  if (bar_test(b, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (bar_test(b, parity)) return true;
    if (*reinterpret_cast<volatile int32_t*>(&sm->failed)) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile int32_t*>(&sm->failed) = 1;
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
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(b))
      : "memory");
}
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Operand descriptor, 128-byte swizzle: start address, leading and stride offsets in
// 16-byte units, version 1.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 |
         (uint64_t)((stride >> 4) & 0x3FFF) << 32 | 1ull << 46 | 2ull << 61;
}
// fp16 x fp16 -> fp32, M = 128, N columns; B's N index contiguous if kTransposed.
template <int N, bool kTransposed>
__device__ __forceinline__ constexpr uint32_t instruction() {
  return 1u << 4 | (kTransposed ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
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

// Keys [lo, hi) that any row of the row tile sees, lo rounded down to 16, and the
// tile's steps (at least one).
struct TileRange {
  int lo, hi, steps;
};
__device__ __forceinline__ TileRange tile_range(const AttendArgs& a, const Request& r, int64_t tile) {
  const int64_t row0 = tile * kTileRows, row1 = min(row0 + kTileRows, r.w * a.G) - 1;
  const int64_t p0 = r.L - r.w + row0 / a.G, p1 = r.L - r.w + row1 / a.G;
  const int64_t lo = a.window ? p0 - a.window + 1 : 0;
  TileRange t;
  t.lo = (int)max((int64_t)0, lo) & ~15;
  t.hi = (int)max((int64_t)0, a.causal ? min(r.L, p1 + 1) : r.L);
  t.steps = t.hi > t.lo ? (t.hi - t.lo + kTileKeys - 1) / kTileKeys : 1;
  return t;
}

// Walks the items (request, kv head, row tile) of a block's share of the steps, the
// same way in every warp.
struct TileWalk {
  long long u, u_end;
  Request req;
  long long head_units;  // steps of one head of the request
  int64_t tiles, tile;
  TileRange range;
  int b, h, s0, s1;      // steps [s0, s1) of the item are this block's

  __device__ __forceinline__ static long long steps_of(const AttendArgs& a, const Request& r,
                                                       int from, int stride) {
    long long x = 0;
    const int64_t n = (r.w * a.G + kTileRows - 1) / kTileRows;
    for (int64_t t = from; t < n; t += stride) x += tile_range(a, r, t).steps;
    return x;
  }
  // Whole-warp: the request's steps of one head.
  __device__ __forceinline__ void enter(const AttendArgs& a, int to) {
    b = to;
    req = request_of(a, b, false);
    tiles = (req.w * a.G + kTileRows - 1) / kTileRows;
    long long x = steps_of(a, req, threadIdx.x & 31, 32);
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
    while (into >= range.steps) {
      into -= range.steps;
      range = tile_range(a, req, ++tile);
    }
    s0 = (int)into;
    s1 = (int)min((long long)range.steps, s0 + (u_end - u));
  }
  __device__ __forceinline__ bool next(const AttendArgs& a) {  // false behind the last item
    u += s1 - s0;
    if (u >= u_end) return false;
    if (++tile == tiles) {
      tile = 0;
      if (++h == a.H) {
        h = 0;
        do enter(a, b + 1);
        while (tiles == 0);
      }
    }
    range = tile_range(a, req, tile);
    s0 = 0;
    s1 = (int)min((long long)range.steps, u_end - u);
    return true;
  }
};

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
constexpr uint32_t kPlus2 = 0x3C003C00u, kMinus2 = 0xBC00BC00u;      // 1, -1
constexpr uint32_t kOffPlus2 = 0xE480E480u, kOffMinus2 = 0x64806480u;  // -1152, 1152

// One block an SM.  Per step of 128 keys a converter warpgroup turns the codes of K
// and V into fp16 operands in shared memory (two stages), one thread issues
//   S_i = Q_i K^T (i = 0, 1: the two halves of 128 rows), O_i += P_i V
// with S and O in TMEM, and a warpgroup for each half turns S_i into P_i: a thread is
// a row.  P_i takes the place of S_i in TMEM as fp16 pairs.  The halves alternate
// (P_0 V, Q_0 K', P_1 V, Q_1 K'), so that one half's exponentials run under the other's
// products.  Scales: the score factor holds the key scale (one for 16 keys); the value
// scale goes into the exponent, p 2^7 scale / vref = 2^(s - m + log2(..)), and the
// row sum takes it out again once in 16 keys, so neither costs work per element.  O is
// rescaled only when a row's maximum rises by more than 2^kSlack or vref changes.
template <int D, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) k_kv_tiles(AttendArgs a) {
  pdl_enter();
  pdl_trigger();
  using L = TileSmem<D>;
  extern __shared__ __align__(16) uint8_t s_tile[];
  const uint32_t base = (smem_addr(s_tile) + 1023) & ~1023u;
  TileSmall* sm = reinterpret_cast<TileSmall*>(s_tile + (base - smem_addr(s_tile)) + L::kSmall);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kTileThreads / 32;

  if (warp == kSoftWarps + kConvWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&sm->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < kTileStages; ++i) {
      bar_init(&sm->k_full[i], 32 * kConvWarps);
      bar_init(&sm->v_full[i], 32 * kConvWarps);
      bar_init(&sm->k_free[i], 1);
      bar_init(&sm->v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm->q_full[i], 128);
      bar_init(&sm->p_full[i], 128);
      bar_init(&sm->s_full[i], 1);
      bar_init(&sm->o_full[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) bar_init(&sm->scales[i], 1);
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
    mine += TileWalk::steps_of(a, r, by_warp ? lane : 0, by_warp ? 32 : 1) * a.H;
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
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sm->sums[i];
    total += sm->sums[i];
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < 1) per = 1;
  const long long u0 = per * blockIdx.x, u_end = min(total, u0 + per);
  {
    // the worker whose requests hold step u0 walks them
    const long long from = by_warp ? before : before + incl - mine;
    const long long to = by_warp ? before + sm->sums[warp] : before + incl;
    if (from <= u0 && u0 < to) {
      long long at = from;
      for (int b = b_lo; b < b_hi; ++b) {
        const Request r = request_of(a, b, false);
        long long x = TileWalk::steps_of(a, r, by_warp ? lane : 0, by_warp ? 32 : 1) * a.H;
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
  const uint32_t tmem = sm->tmem;
  const bool any = u0 < u_end;
  TileWalk walk;
  if (any) walk.start(a, sm->b, u0 - sm->before, u0, u_end);

  if (!any) {
    // no steps here
  } else if (warp < kSoftWarps) {
    // ================================================================ softmax
    const int half = warp >> 2;
    const int at_row = (warp & 3) * 32 + lane;  // of the half = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + half * 128 + lanes, t_o = tmem + 256 + half * D + lanes;
    uint32_t n_s = 0, n_o = 0, n_k = 0;  // s_full and o_full phases, steps so far
    PartHead head = {0, 0, 0, -1};
    bool ok = true;
    do {
      const Request req = walk.req;
      const int64_t rows = req.w * a.G, row0 = walk.tile * kTileRows + half * 128;
      const int n_steps = walk.s1 - walk.s0;
      const bool begins = walk.s0 == 0, ends = walk.s1 == walk.range.steps;
      if (begins && !ends) {
        head.b = walk.b;
        head.h = walk.h;
        head.tile = (int)walk.tile;
        head.last = (int)((walk.u + walk.range.steps - 1) / per);
      }
      if (row0 >= rows) {  // this half of the tile is empty
        n_k += n_steps;
        continue;
      }
      const int64_t row = row0 + at_row;
      const bool real = row < rows;
      const int64_t t = real ? row / a.G : 0;
      const int hq = walk.h * a.G + (int)(real ? row % a.G : 0);
      // ---- the row's queries, scaled by a power of two, as fp16 in shared memory
      const T* q = static_cast<const T*>(a.q) + (req.start + t) * a.qsn + hq * a.qsh;
      uint32_t amax = 0;
      if (real) {
#pragma unroll
        for (int d = 0; d < D; d += 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + d));
          const T* x = reinterpret_cast<const T*>(&v);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            amax = max(amax, __float_as_uint((float)x[e]) & 0x7FFFFFFFu);
        }
      }
      const float qfac = copysignf(row_factor(amax), a.scale_log2);
      const float inv = __fdiv_rn(a.scale_log2, qfac);
      const uint32_t q_at = base + L::kQ + half * L::kOperand + at_row * 128;
#pragma unroll
      for (int d = 0; d < D; d += 8) {
        uint4 y = make_uint4(0, 0, 0, 0);
        if (real && qfac == qfac) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q + d));
          const T* x = reinterpret_cast<const T*>(&v);
          y.x = half2_bits(__fmul_rn((float)x[0], qfac), __fmul_rn((float)x[1], qfac));
          y.y = half2_bits(__fmul_rn((float)x[2], qfac), __fmul_rn((float)x[3], qfac));
          y.z = half2_bits(__fmul_rn((float)x[4], qfac), __fmul_rn((float)x[5], qfac));
          y.w = half2_bits(__fmul_rn((float)x[6], qfac), __fmul_rn((float)x[7], qfac));
        }
        const uint32_t to = q_at + (d / 64) * L::kPlane + (((d % 64) * 2) ^ ((at_row & 7) << 4));
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(y.x), "r"(y.y), "r"(y.z),
                     "r"(y.w)
                     : "memory");
      }
      proxy_fence();
      bar_arrive(&sm->q_full[half]);

      const int64_t pos = req.L - req.w + t;
      const int hi = real ? (int)max((int64_t)0, a.causal ? min(req.L, pos + 1) : req.L) : 0;
      const int lo = a.window ? (int)max((int64_t)0, pos - a.window + 1) : 0;
      float m = -CUDART_INF_F, sum = 0.f;
      float vref = 0.f, lref = 0.f;  // power of two above the value scales, its log2
      for (int j = 0; j < n_steps && ok; ++j, ++n_k) {
        const int key = walk.range.lo + (walk.s0 + j) * kTileKeys;
        const int slot = n_k % kScaleSlots;
        ok = bar_wait(&sm->scales[slot], (n_k / kScaleSlots) & 1, sm, a.status) &&
             bar_wait(&sm->s_full[half], n_s & 1, sm, a.status);
        if (!__all_sync(kAll, ok)) {
          ok = false;
          break;
        }
        ++n_s;
        tc_fence_after();
        const float* ks = sm->ks[slot];
        const float* vs = sm->vs[slot];
        const uint32_t none = sm->hidden[slot];
        // does every row of the warp see every key?  (real rows; the others' results
        // are not used)
        const bool hide =
            none || __any_sync(kAll, real && (key + kTileKeys > hi || key < lo));
        // ---- largest score
        float mx = -CUDART_INF_F, va = 0.f;
        uint32_t x[2][32];
        tmem_load32(t_s, x[0]);
#pragma unroll
        for (int cnk = 0; cnk < 4; ++cnk) {
          uint32_t (&y)[32] = x[cnk & 1];
          tmem_loaded(y);
          if (cnk < 3) tmem_load32(t_s + (cnk + 1) * 32, x[(cnk + 1) & 1]);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float f = __fmul_rn(inv, fabsf(ks[cnk * 2 + g]));
            const float v = fabsf(vs[cnk * 2 + g]);
            if (v < CUDART_INF_F) va = fmaxf(va, v);
            float best = -CUDART_INF_F;
            if (hide) {
              const int k0 = key + cnk * 32 + g * 16;
              const int to = none >> (cnk * 2 + g) & 1 ? lo : hi;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (k0 + e < to && k0 + e >= lo) best = fmaxf(best, __uint_as_float(y[g * 16 + e]));
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) best = fmaxf(best, __uint_as_float(y[g * 16 + e]));
            }
            if (best > -CUDART_INF_F) mx = fmaxf(mx, __fmul_rn(best, f));
          }
        }
        const bool vup = va > vref;
        if (__any_sync(kAll, mx > m + kSlack) || vup) {
          float beta = 1.f;
          if (vup) {
            const uint32_t e = (__float_as_uint(va) >> 23) + 1;
            const float to = __uint_as_float((e > 254 ? 254 : e) << 23);
            beta = __fdiv_rn(vref, to);
            vref = to;
            lref = (float)((int)(e > 254 ? 254 : e) - 127);
          }
          const float to = fmaxf(m, mx);
          const float alpha = to == m ? 1.f : exp2_fast(m - to);
          m = to;
          sum = __fmul_rn(sum, alpha);
          if (j > 0) {
            const float g = __fmul_rn(alpha, beta);
#pragma unroll
            for (int d = 0; d < D; d += 32) {
              tmem_load32(t_o + d, x[0]);
              tmem_loaded(x[0]);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[0][e] = __float_as_uint(__fmul_rn(__uint_as_float(x[0][e]), g));
              tmem_store32(t_o + d, x[0]);
            }
            tmem_stored();
          }
        }
        // ---- weights.  Scores beyond 2^20 in log2 units are rounded like the maximum
        // before it is taken off; below, one fma does.
        const float top = m == -CUDART_INF_F ? 0.f : m;
        const bool big = __any_sync(kAll, fabsf(top) > 1048576.f);
        tmem_load32(t_s, x[0]);
#pragma unroll
        for (int cnk = 0; cnk < 4; ++cnk) {
          uint32_t (&y)[32] = x[cnk & 1];
          tmem_loaded(y);
          if (cnk < 3) tmem_load32(t_s + (cnk + 1) * 32, x[(cnk + 1) & 1]);
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float f = __fmul_rn(inv, fabsf(ks[cnk * 2 + g]));
            // log2 of 2^7 scale / vref; far below, the weights vanish in fp16 anyway
            float lp = __fadd_rn(__fsub_rn(__log2f(fabsf(vs[cnk * 2 + g])), lref), 7.f);
            lp = lp < -60.f ? -60.f : lp;
            const float off = __fsub_rn(lp, top);
            float s16 = 0.f;
            float p[16];
            if (big) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                p[e] = exp2_fast(__fadd_rn(
                    __fsub_rn(__fmul_rn(__uint_as_float(y[g * 16 + e]), f), top), lp));
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                p[e] = exp2_fast(__fmaf_rn(__uint_as_float(y[g * 16 + e]), f, off));
            }
            if (hide) {
              const int k0 = key + cnk * 32 + g * 16;
              const int to = none >> (cnk * 2 + g) & 1 ? lo : hi;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!(k0 + e < to && k0 + e >= lo)) p[e] = 0.f;
            }
            float s4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s4[e] = __fadd_rn(__fadd_rn(p[e], p[e + 4]), __fadd_rn(p[e + 8], p[e + 12]));
            s16 = __fadd_rn(__fadd_rn(s4[0], s4[1]), __fadd_rn(s4[2], s4[3]));
            if (s16 != 0.f) sum = __fmaf_rn(s16, exp2_fast(-lp), sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) pk[g * 8 + e] = half2_bits(p[2 * e], p[2 * e + 1]);
          }
          tmem_store16(t_s + cnk * 16, pk);
        }
        tmem_stored();
        tc_fence_before();
        bar_arrive(&sm->p_full[half]);
      }
      if (!ok) break;
      // ---- the row's result
      ok = bar_wait(&sm->o_full[half], n_o & 1, sm, a.status);
      if (!__all_sync(kAll, ok)) {
        ok = false;
        break;
      }
      ++n_o;
      tc_fence_after();
      const float unit = __fmul_rn(vref, 1.f / kWeightScale);
      const bool whole = begins && ends;
      const float g = whole ? (sum == 0.f ? 0.f : __fdiv_rn(unit, sum)) : unit;
      float* part = a.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kTileRows * (D + 2);
      const int prow = half * 128 + at_row;
#pragma unroll
      for (int d = 0; d < D; d += 32) {
        uint32_t x[32];
        tmem_load32(t_o + d, x);
        tmem_loaded(x);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          // a row that saw no key: 0, whatever the hidden blocks hold
          o[e] = sum == 0.f ? 0.f : __fmul_rn(__uint_as_float(x[e]), g);
        if (real) {
          if (whole)
            store_row<T>(static_cast<T*>(a.out) + (req.start + t) * a.osn + hq * a.osh + d, o);
          else
            store_row<float>(part + prow * D + d, o);
        }
      }
      if (real) {
        if (!whole)
          *reinterpret_cast<float2*>(part + kTileRows * D + prow * 2) = make_float2(m, sum);
        else if (a.lse)
          a.lse[(req.start + t) * a.Hq + hq] =
              sum == 0.f ? -CUDART_INF_F : __fmul_rn(m + log2f(sum), 0.6931471805599453f);
      }
      tc_fence_before();
    } while (walk.next(a));
    if (tid == 0) a.heads[blockIdx.x] = head;
  } else if (warp < kSoftWarps + kConvWarps) {
    // ================================================================ converters
    const int ct = tid - 32 * kSoftWarps, col = ct & 7, row_in = ct >> 3;
    constexpr int kPlanes = D / 64;
    const int bs = 1 << a.bs_log;
    uint32_t n_k = 0;
    bool ok = true;
    do {
      const int n_steps = walk.s1 - walk.s0;
      const int32_t* row_table = a.table + (int64_t)walk.b * a.max_blocks;
      const int8_t* kb = a.k + (((int64_t)walk.h << a.bs_log) + row_in) * D + col * 8;
      const int8_t* vb = a.v + (((int64_t)walk.h << a.bs_log) + row_in) * D + col * 8;
      const int64_t block_bytes = ((int64_t)a.H << a.bs_log) * D;
      const int key0 = walk.range.lo + walk.s0 * kTileKeys;
      // lane g < 8: block id (-1: none, its keys are hidden) and scales of 16-key group g
      auto look_up = [&](int j, int32_t& id, float& ks, float& vs) {
        id = -1;
        ks = vs = 0.f;
        const int key = key0 + j * kTileKeys + lane * 16;
        if (lane < kGroups && j < n_steps && key < walk.range.hi) {
          id = __ldg(row_table + (key >> a.bs_log));
          if (id < 0 || id >= a.num_blocks) {
            id = -1;
            set_status(a.status, kStBadBlock);
          } else {
            ks = __ldg(a.ks + (int64_t)id * a.H + walk.h);
            vs = __ldg(a.vs + (int64_t)id * a.H + walk.h);
          }
        }
      };
      auto load = [&](const int8_t* from, int j, int32_t id_l, uint2 (&w)[kGroups][kPlanes]) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const int32_t id = __shfl_sync(kAll, id_l, g);
          const int key = key0 + j * kTileKeys + g * 16;
          const int8_t* p = from + id * block_bytes + (key & (bs - 1)) * D;
#pragma unroll
          for (int pl = 0; pl < kPlanes; ++pl) {
            w[g][pl] = make_uint2(0, 0);
            if (id >= 0) w[g][pl] = __ldg(reinterpret_cast<const uint2*>(p + pl * 64));
          }
        }
      };
      auto store = [&](uint32_t to, float scale_l, const uint2 (&w)[kGroups][kPlanes]) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          // a negative scale (no append gives one) goes into the codes' sign
          const bool neg = __shfl_sync(kAll, scale_l, g) < 0.f;
          const uint32_t sign2 = neg ? kMinus2 : kPlus2, off2 = neg ? kOffMinus2 : kOffPlus2;
          const int row = g * 16 + row_in;
          const uint32_t at = to + row * 128 + ((col * 16) ^ ((row & 7) << 4));
#pragma unroll
          for (int pl = 0; pl < kPlanes; ++pl) {
            const uint4 y = codes_to_half8(w[g][pl], sign2, off2);
            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at + pl * L::kPlane), "r"(y.x),
                         "r"(y.y), "r"(y.z), "r"(y.w)
                         : "memory");
          }
        }
      };
      int32_t id, id_n;
      float ks, vs, ks_n, vs_n;
      uint2 wk[kGroups][kPlanes], wv[kGroups][kPlanes];
      look_up(0, id, ks, vs);
      load(kb, 0, id, wk);
      for (int j = 0; j < n_steps && ok; ++j, ++n_k) {
        const int stage = n_k % kTileStages;
        const uint32_t again = ((n_k / kTileStages) & 1) ^ 1;
        load(vb, j, id, wv);
        look_up(j + 1, id_n, ks_n, vs_n);
        ok = bar_wait(&sm->k_free[stage], again, sm, a.status);
        if (!__all_sync(kAll, ok)) {
          ok = false;
          break;
        }
        store(base + L::kK + stage * L::kOperand, ks, wk);
        if (warp == kSoftWarps) {
          const int slot = n_k % kScaleSlots;
          const uint32_t none = __ballot_sync(kAll, id < 0) & ((1u << kGroups) - 1);
          if (lane < kGroups) {
            sm->ks[slot][lane] = ks;
            sm->vs[slot][lane] = vs;
          }
          if (lane == 0) sm->hidden[slot] = none;
          __syncwarp();
          if (lane == 0) bar_arrive(&sm->scales[slot]);
        }
        proxy_fence();
        bar_arrive(&sm->k_full[stage]);
        if (j + 1 < n_steps) load(kb, j + 1, id_n, wk);
        ok = bar_wait(&sm->v_free[stage], again, sm, a.status);
        if (!__all_sync(kAll, ok)) {
          ok = false;
          break;
        }
        store(base + L::kV + stage * L::kOperand, vs, wv);
        proxy_fence();
        bar_arrive(&sm->v_full[stage]);
        id = id_n;
        ks = ks_n;
        vs = vs_n;
      }
    } while (ok && walk.next(a));
  } else {
    // ================================================================ products
    uint32_t n_k = 0, n_q[2] = {0, 0}, n_p[2] = {0, 0};
    constexpr uint32_t kScores = instruction<kTileKeys, false>(), kOut = instruction<D, true>();
    bool ok = true;
    do {
      const int n_steps = walk.s1 - walk.s0;
      const int64_t rows = walk.req.w * a.G - walk.tile * kTileRows;
      const int halves = rows > 128 ? 2 : 1;
      if (lane == 0) {
        auto scores = [&](int i, uint32_t step) {
          const uint32_t q = base + L::kQ + i * L::kOperand;
          const uint32_t k = base + L::kK + (step % kTileStages) * L::kOperand;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t at = (kk / 4) * L::kPlane + (kk % 4) * 32;
            mma_ss(tmem + i * 128, operand(q + at, 16, 1024), operand(k + at, 16, 1024), kScores,
                   kk > 0);
          }
          tc_commit(&sm->s_full[i]);
        };
        for (int i = 0; i < halves && ok; ++i)
          ok = bar_wait(&sm->q_full[i], n_q[i]++ & 1, sm, a.status);
        if (ok)
          ok = bar_wait(&sm->k_full[n_k % kTileStages], (n_k / kTileStages) & 1, sm, a.status);
        if (ok) {
          tc_fence_after();
          for (int i = 0; i < halves; ++i) scores(i, n_k);
          tc_commit(&sm->k_free[n_k % kTileStages]);
        }
        for (int j = 0; j < n_steps && ok; ++j, ++n_k) {
          const int stage = n_k % kTileStages;
          ok = bar_wait(&sm->v_full[stage], (n_k / kTileStages) & 1, sm, a.status);
          for (int i = 0; i < halves && ok; ++i) {
            ok = bar_wait(&sm->p_full[i], n_p[i]++ & 1, sm, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t v = base + L::kV + stage * L::kOperand;
#pragma unroll
            for (int kk = 0; kk < kTileKeys / 16; ++kk)
              mma_ts(tmem + 256 + i * D, tmem + i * 128 + kk * 8,
                     operand(v + kk * 2048, L::kPlane, 1024), kOut, j > 0 || kk > 0);
            if (i == halves - 1) tc_commit(&sm->v_free[stage]);
            if (j == n_steps - 1) {
              tc_commit(&sm->o_full[i]);
            } else {
              if (i == 0) {
                const uint32_t nx = n_k + 1;
                ok = bar_wait(&sm->k_full[nx % kTileStages], (nx / kTileStages) & 1, sm, a.status);
                if (!ok) break;
                tc_fence_after();
              }
              scores(i, n_k + 1);
              if (i == halves - 1) tc_commit(&sm->k_free[(n_k + 1) % kTileStages]);
            }
          }
        }
      }
      ok = __shfl_sync(kAll, (int)ok, 0) != 0;
    } while (ok && walk.next(a));
  }
  if (!any && tid == 0) {
    const PartHead none = {0, 0, 0, -1};
    a.heads[blockIdx.x] = none;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kConvWarps)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

}  // namespace mpzch_kv
