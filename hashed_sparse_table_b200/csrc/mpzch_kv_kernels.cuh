// Device code of the history cache: block tables and slots, the int8 append,
// and attention for few rows per request (include/mpzch.h, "History cache").
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "mpzch_device.cuh"

namespace mpzch_kv {

using namespace mpzch;

constexpr int kStBadLen = 32, kStNoBlock = 64, kStBadBlock = 128;
constexpr unsigned kAll = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------
// Block tables and slots.
// ---------------------------------------------------------------------------
struct TablesArgs {
  const int32_t *cached, *news;
  int B, bs_log;
  const int32_t* free_blocks;
  int64_t n_free;
  const long long* free_count;
  int32_t* table;
  int max_blocks;
  int32_t *cu, *seq;
  long long* slots;
  int64_t n_slots;
  long long* free_out;
  int32_t* status;
};

// Inclusive scan of one value per thread over the block; `total` gets the sum.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kAll, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // s_warp may still be read from the previous scan
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = 0, sum = 0;
  long long w = lane < nw ? s_warp[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kAll, w, d);
    if (lane >= d) w += y;
  }
  before = __shfl_sync(kAll, w, (warp + 31) & 31);
  sum = __shfl_sync(kAll, w, 31);
  total = sum;
  return x + (warp ? before : 0);
}

// First index in the non-decreasing s[0..n) whose value is > x (n if none).
__device__ __forceinline__ int first_above(const int32_t* s, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One launch.  Every block scans all requests (at most 16,384: two ints each,
// from L2) into shared memory and then writes its share of the rows, of the new
// table entries and of the lengths, so no block waits for another.  Bound by the
// latency of its few dependent loads: 256 requests of one token 5.7 us a call in a
// graph; 4,096 requests with 0.6 million new rows (5.8 MB) 15.8 us alone and cold, below
// the 16.7 us that a caller needs to issue the call and allocate its outputs.
__global__ void __launch_bounds__(1024) k_kv_tables(TablesArgs a) {
  pdl_enter();
  extern __shared__ int32_t s_dyn[];
  __shared__ long long s_warp[32];
  int32_t* s_end = s_dyn;          // rows up to and with request b
  int32_t* s_upto = s_dyn + a.B;   // blocks needed up to and with request b
  constexpr long long kTop = 0x7FFFFFFFll;
  const int bs = 1 << a.bs_log, tid = threadIdx.x, nt = blockDim.x;
  long long count = *a.free_count;
  count = count < 0 ? 0 : count > a.n_free ? a.n_free : count;
  long long tok0 = 0, need0 = 0;
  int bits = 0;
  for (int base = 0; base < a.B; base += nt * 4) {
    const int b0 = base + tid * 4;
    long long c[4], w[4], sum = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = b0 + i < a.B;
      c[i] = in ? a.cached[b0 + i] : 0;
      w[i] = in ? a.news[b0 + i] : 0;
      sum += w[i] > 0 ? w[i] : 0;
    }
    long long end = block_scan(sum, s_warp, total) - sum + tok0;
    tok0 += total;
    long long need[4];
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      end += w[i] > 0 ? w[i] : 0;
      const long long all = (c[i] + w[i] + bs - 1) >> a.bs_log;
      const bool bad = c[i] < 0 || w[i] < 0 || all > a.max_blocks || end > a.n_slots;
      if (bad) bits |= kStBadLen;
      need[i] = bad ? 0 : all - ((c[i] + bs - 1) >> a.bs_log);
      sum += need[i];
      if (b0 + i < a.B) s_end[b0 + i] = (int32_t)(end < kTop ? end : kTop);
    }
    long long upto = block_scan(sum, s_warp, total) - sum + need0;
    need0 += total;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      upto += need[i];
      if (need[i] > 0 && upto > count) bits |= kStNoBlock;
      if (b0 + i < a.B) s_upto[b0 + i] = (int32_t)(upto < kTop ? upto : kTop);
    }
  }
  __syncthreads();
  const int gtid = blockIdx.x * nt + tid, gthreads = gridDim.x * nt;
  // blocks given out: the largest s_upto that the list holds
  const int served = first_above(s_upto, a.B, (int)count);
  const int given = served ? s_upto[served - 1] : 0;
  if (blockIdx.x == 0) {
    if (bits) set_status(a.status, bits);
    if (tid == 0) {
      a.cu[0] = 0;
      *a.free_out = count - given;
    }
  }
  // lengths
  for (int b = gtid; b < a.B; b += gthreads) {
    const long long c = a.cached[b], w = a.news[b];
    const long long all = (c + w + bs - 1) >> a.bs_log;
    const bool bad = c < 0 || w < 0 || all > a.max_blocks || s_end[b] > a.n_slots;
    const int32_t before = b ? s_upto[b - 1] : 0;
    const bool ok = !bad && (s_upto[b] == before || s_upto[b] <= count);
    a.cu[b + 1] = s_end[b];
    a.seq[b] = (int32_t)(ok ? c + w : c > 0 ? c : 0);
  }
  // new table entries: entry e of those given out belongs to the first request
  // with s_upto > e
  for (int64_t e = gtid; e < given; e += gthreads) {
    const int b = first_above(s_upto, served, (int)e);
    const int before = b ? s_upto[b - 1] : 0;
    const long long old = ((long long)a.cached[b] + bs - 1) >> a.bs_log;
    a.table[(int64_t)b * a.max_blocks + old + (e - before)] = a.free_blocks[count - 1 - e];
  }
  // slots, 4 rows a thread
  const int64_t rows = tok0 < a.n_slots ? tok0 : a.n_slots;
  for (int64_t i0 = (int64_t)gtid * 4; i0 < a.n_slots; i0 += (int64_t)gthreads * 4) {
    long long out[4] = {-1, -1, -1, -1};
    if (i0 < rows) {
      int b = first_above(s_end, a.B, (int)i0);
      bool ok = false;
      long long c = 0, start = 0, old = 0, held = -1;
      int32_t before = 0, next = 0;
      bool fresh = true;
      long long blk = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = i0 + i;
        if (r < rows) {
          while (r >= s_end[b]) {
            ++b;
            fresh = true;
          }
          if (fresh) {
            c = a.cached[b];
            start = b ? s_end[b - 1] : 0;
            old = (c + bs - 1) >> a.bs_log;
            before = b ? s_upto[b - 1] : 0;
            next = s_upto[b];
            const long long all = (c + (s_end[b] - start) + bs - 1) >> a.bs_log;
            ok = c >= 0 && all <= a.max_blocks && s_end[b] <= a.n_slots &&
                 (next == before || next <= count);
            held = -1;
            fresh = false;
          }
          if (ok) {
            const long long pos = c + (r - start), j = pos >> a.bs_log;
            if (j != held) {
              blk = j < old ? a.table[(int64_t)b * a.max_blocks + j]
                            : a.free_blocks[count - 1 - (before + (j - old))];
              held = j;
            }
            out[i] = (blk << a.bs_log) + (pos & (bs - 1));
          }
        }
      }
    }
    if (i0 + 4 <= a.n_slots && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
      reinterpret_cast<longlong2*>(a.slots + i0)[0] = make_longlong2(out[0], out[1]);
      reinterpret_cast<longlong2*>(a.slots + i0)[1] = make_longlong2(out[2], out[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < a.n_slots) a.slots[i0 + i] = out[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Append.
// ---------------------------------------------------------------------------
struct AppendArgs {
  const void* x[2];        // k, v
  int64_t sn[2], sh[2];    // element strides of rows and heads
  int64_t n;
  const long long* slots;
  int8_t* cache[2];
  float* scale[2];
  int64_t num_blocks;
  int bs_log, H;
  int rows_per_warp;       // 1..32
  int32_t* status;
};

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(lo), "f"(hi));
  return x;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t x;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(a), "l"(b), "l"(c));
  return x;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t x;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(a), "l"(b));
  return x;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float x;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(x) : "f"(a), "f"(b), "f"(c));
  return x;
}
// 16 consecutive values of a row as they come: 2 (fp32: 4) 16-byte vectors.
template <typename T>
struct Raw16 {
  static constexpr int kVec = (int)sizeof(T);
  uint4 v[kVec];
};

template <typename T>
__device__ __forceinline__ void load_raw(const T* p, Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < Raw16<T>::kVec; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}

// Values 2i and 2i + 1.
template <typename T>
__device__ __forceinline__ uint64_t raw_pair(const Raw16<T>& r, int i) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
  if constexpr (sizeof(T) == 4) {
    return pair(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else if constexpr (__is_same(T, __nv_bfloat16)) {
    return pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    return pair(f.x, f.y);
  }
}

// Largest |x| so far, as the bits of an fp32 (a) or of two 16-bit numbers: for
// non-negative floats the order of the bits is the order of the values, with every NaN
// above infinity.
template <typename T>
__device__ __forceinline__ uint32_t absmax_raw(const Raw16<T>& r, uint32_t a) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
#pragma unroll
  for (int i = 0; i < 4 * Raw16<T>::kVec; ++i)
    a = sizeof(T) == 4 ? max(a, w[i] & 0x7FFFFFFFu) : __vmaxu2(a, w[i] & 0x7FFF7FFFu);
  return a;
}
// The same as an fp32.
template <typename T>
__device__ __forceinline__ float absmax_value(uint32_t a) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(a);
  } else {
    const uint32_t top = max(a & 0xFFFFu, a >> 16);
    if constexpr (__is_same(T, __nv_bfloat16)) return __uint_as_float(top << 16);
    return __half2float(__ushort_as_half((unsigned short)top));
  }
}

// rne(fl(x / s)) of 16 values (as pairs).  16-bit inputs lie on the halves between two
// codes often (x = a / 2 gives 63.5), so the quotient itself is formed, in packed
// arithmetic: by Markstein's theorem ("Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) q' = fma(fma(-q, s, x), rcp, q) with the correctly rounded
// reciprocal rcp is the correctly rounded quotient when q is within an ulp of it, which
// the first correction sees to (x rcp is within 1.5).  That needs s in the middle of the
// exponent range; elsewhere (uniformly for a run) the values are divided.  The integer
// then comes out of adding 1.5 2^23, in the low byte of the sum.  A run's own values give
// quotients of 127 at most; held ones (kCut; `near`: the old scale is within 2^20 s) pass
// it where the old scale is negative or a code is -128, neither of which an append leaves.
template <bool kCut>
__device__ __forceinline__ uint4 codes16(const uint64_t (&x)[8], float s, float rcp, bool near) {
  uint32_t b[16];
  auto cut = [](float q) { return fminf(fmaxf(q, -127.f), 127.f); };
  if (s >= 0x1p-80f && s <= 0x1p100f && near) {
    const uint64_t r2 = pair(rcp, rcp), s2 = pair(-s, -s), magic = pair(kRoundMagic, kRoundMagic);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint64_t q = mul2(x[i], r2);
      q = fma2(fma2(q, s2, x[i]), r2, q);
      q = fma2(fma2(q, s2, x[i]), r2, q);
      float lo, hi;
      if constexpr (kCut) {
        unpair(q, lo, hi);
        q = pair(cut(lo), cut(hi));
      }
      unpair(add2(q, magic), lo, hi);
      b[2 * i] = __float_as_uint(lo);
      b[2 * i + 1] = __float_as_uint(hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float lo, hi;
      unpair(x[i], lo, hi);
      b[2 * i] = rne_small(cut(__fdiv_rn(lo, s)));
      b[2 * i + 1] = rne_small(cut(__fdiv_rn(hi, s)));
    }
  }
  return make_uint4(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]),
                    pack4(b[8], b[9], b[10], b[11]), pack4(b[12], b[13], b[14], b[15]));
}

// A group of W warps takes rows_per_warp rows of the batch for one head of one cache and
// works through the runs that begin there.  A lane handles 16 values of a token, a warp
// 4 x 32 * 16 / D tokens, all of its loads in flight together; W is what a whole block
// of tokens needs, so every value is read once and waits in registers for the maximum.
// A long batch is near HBM and near its issue slots: 104 thousand bf16 tokens x 8 heads x
// 128 in 32-token blocks (849 MB) 177 us a call, 4.8 TB/s, 0.73 of the measured copy rate,
// instructions issued in 0.55 of the cycles; a warp's runs follow one another, so each
// one's loads wait in the open.  31 thousand fp32 tokens x 4 heads x 128 in 64-token blocks
// (176 MB) 44 us, 4.0 TB/s, where a group has few runs.  256 single tokens of 8
// heads x 64 take 3.9 us in a graph.  Measured and dropped: half the passes kept and
// twice the warps (the per-run work doubled: 217 -> 247 us), and the export's test for
// nearly half-way products, which 16-bit values fail in nearly every warp (260 us).
constexpr int kAppendKeep = 4;
__host__ __device__ constexpr int append_warps(int D, int bs) {
  return bs * D / 512 / kAppendKeep > 1 ? bs * D / 512 / kAppendKeep : 1;
}

template <typename T, int D, int W>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 3) k_kv_append(AppendArgs a) {
  pdl_enter();
  constexpr int kLanes = D / 16, kTok = 32 / kLanes, kKeep = kAppendKeep;
  __shared__ uint32_t s_max[2][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp / W, wi = warp % W;
  const int bs = 1 << a.bs_log;
  const int sub = lane % kLanes, tok = wi * (kKeep * kTok) + lane / kLanes;
  // blocks of one head and cache each, so that no task number has to be divided
  const int h = blockIdx.x >> 1, which = blockIdx.x & 1;
  const T* __restrict__ src = static_cast<const T*>(which ? a.x[1] : a.x[0]);
  const int64_t sn = which ? a.sn[1] : a.sn[0];
  src += h * (which ? a.sh[1] : a.sh[0]) + sub * 16;
  int8_t* cache = (which ? a.cache[1] : a.cache[0]) + ((int64_t)h << a.bs_log) * D + sub * 16;
  float* scale = (which ? a.scale[1] : a.scale[0]) + h;
  const int64_t block_bytes = ((int64_t)a.H << a.bs_log) * D;
  uint32_t turn = 0;
  // slots of this lane's row and of the one before, asked for one round ahead
  long long slot_n = -1, prev_n = -2;
  auto ask = [&](int64_t row0) {
    const int64_t mine = row0 + lane;
    const bool in = lane < a.rows_per_warp && mine < a.n;
    slot_n = in ? __ldg(a.slots + mine) : -1;
    prev_n = in && mine > 0 ? __ldg(a.slots + mine - 1) : -2;
  };
  const int64_t stride = (int64_t)gridDim.y * (8 / W) * a.rows_per_warp;
  int64_t row0 = ((int64_t)blockIdx.y * (8 / W) + group) * a.rows_per_warp;
  ask(row0);
  for (; row0 < a.n; row0 += stride) {
    const long long slot_l = slot_n, prev_l = prev_n;
    ask(row0 + stride);
    const bool bad = slot_l >= 0 && (slot_l >> a.bs_log) >= a.num_blocks;
    if (bad) set_status(a.status, kStBadBlock);
    unsigned heads = __ballot_sync(
        kAll, slot_l >= 0 && !bad && (slot_l != prev_l + 1 || (slot_l & (bs - 1)) == 0));
    while (heads) {
      const int l = __ffs(heads) - 1;
      heads &= heads - 1;
      const long long slot = __shfl_sync(kAll, slot_l, l);
      const int64_t row = row0 + l, blk = slot >> a.bs_log;
      const int o = (int)(slot & (bs - 1));
      int len = 0;
      for (int d = 0; d < bs - o; d += 32) {
        const bool next = d + lane < bs - o && row + d + lane < a.n &&
                          __ldg(a.slots + row + d + lane) == slot + d + lane;
        const unsigned miss = ~__ballot_sync(kAll, next);
        len += miss ? __ffs(miss) - 1 : 32;
        if (miss) break;
      }
      const T* p = src + row * sn;
      Raw16<T> x[kKeep];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (i * kTok + tok < len) load_raw(p + (int64_t)(i * kTok + tok) * sn, x[i]);
      float* sp = scale + blk * a.H;
      const float before = o > 0 ? *sp : 0.f;
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (i * kTok + tok < len) amax = absmax_raw(x[i], amax);
      float top = absmax_value<T>(amax);  // not negative: its bits are in order
      top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(top)));
      if constexpr (W > 1) {
        // the slot of two runs ago has been read by every warp: this barrier was between
        uint32_t* s = s_max[turn++ & 1];
        if (lane == 0) s[warp] = __float_as_uint(top);
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(1 + group), "n"(32 * W) : "memory");
        uint32_t t = s[group * W];
#pragma unroll
        for (int i = 1; i < W; ++i) t = max(t, s[group * W + i]);
        top = __uint_as_float(t);
      }
      const float own = __fdiv_rn(top, 127.0f);
      // the larger one; a NaN on either side stays
      const float s = own != own ? own : (before >= own || before != before) ? before : own;
      const bool usable = s > 0.f && s < CUDART_INF_F;
      const float rcp = usable ? __frcp_rn(s) : 0.f;
      int8_t* base = cache + blk * block_bytes;
      if (o > 0 && s != before && (s == s || before == before)) {
        for (int i = wi * kTok + lane / kLanes; i < o; i += W * kTok) {
          uint4* c = reinterpret_cast<uint4*>(base + (int64_t)i * D);
          const uint4 v = *c;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint64_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            y[j] = pair(__fmul_rn((float)(int8_t)(w[j / 2] >> (16 * (j % 2))), before),
                        __fmul_rn((float)(int8_t)(w[j / 2] >> (16 * (j % 2) + 8)), before));
          *c = usable ? codes16<true>(y, s, rcp, fabsf(before) <= __fmul_rn(s, 0x1p20f))
                      : make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (i * kTok + tok < len) {
          uint64_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = raw_pair(x[i], j);
          *reinterpret_cast<uint4*>(base + (int64_t)(o + i * kTok + tok) * D) =
              usable ? codes16<false>(y, s, rcp, true) : make_uint4(0, 0, 0, 0);
        }
      __syncwarp();  // every lane has read the old scale (W > 1: and every warp)
      if (wi == 0 && lane == 0) *sp = s;
    }
  }
}

}  // namespace mpzch_kv
