// Attention over the history cache for few rows per request (decode steps,
// drafted tokens), and for every shape the tile kernel does not take.
#pragma once
#include "mpzch_kv_kernels.cuh"

namespace mpzch_kv {

constexpr int kRowTile = 16;    // query rows (token, head of the group) of one tile
constexpr int kStepKeys = 64;   // keys of one step of a block: 16 for each of 4 warps
constexpr int kRowWarps = 4;
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
  float* lse;
  int32_t* status;
  int64_t most_rows;  // requests with more rows are left to the tile kernel
  int min_steps;      // steps that a block takes at least
  struct PartHead* heads;
  float* parts;       // [block][2][kRowTile][D + 2]
};

// What a block of k_kv_rows leaves for k_kv_join: the item that begins in the
// block and ends in block `last` (< 0: none).
struct PartHead {
  int32_t b, h, tile, last;
};

struct Request {
  int64_t start;  // first row of the batch
  int64_t w;      // rows (new tokens)
  int64_t L;      // keys
};

__device__ __forceinline__ Request request_of(const AttendArgs& a, int b, bool report) {
  Request r;
  const int64_t s0 = a.cu[b], e0 = a.cu[b + 1], l0 = a.seq[b];
  const int64_t most = (int64_t)a.max_blocks << a.bs_log;
  const int64_t s = s0 < 0 ? 0 : s0 > a.n ? a.n : s0;
  const int64_t e = e0 < s ? s : e0 > a.n ? a.n : e0;
  const int64_t l = l0 < 0 ? 0 : l0 > most ? most : l0;
  if (report && (s != s0 || e != e0 || l != l0)) set_status(a.status, kStBadLen);
  r.start = s;
  r.w = e - s;
  r.L = l;
  return r;
}

// Keys [lo, hi) that the request's rows see between them, lo rounded down to 16.
__device__ __forceinline__ int64_t first_key(const AttendArgs& a, const Request& r) {
  if (!a.window) return 0;
  const int64_t lo = r.L - r.w - a.window + 1;
  return lo > 0 ? lo & ~(int64_t)15 : 0;
}

// Steps of one (head, row tile) of the request; every such item has the same
// number, at least one.
__device__ __forceinline__ int64_t item_steps(const AttendArgs& a, const Request& r) {
  const int64_t keys = r.L - first_key(a, r);
  return keys > kStepKeys ? (keys + kStepKeys - 1) / kStepKeys : 1;
}

__device__ __forceinline__ int64_t row_tiles(const AttendArgs& a, const Request& r) {
  return r.w * a.G > a.most_rows ? 0 : (r.w * a.G + kRowTile - 1) / kRowTile;
}

__device__ __forceinline__ int64_t request_units(const AttendArgs& a, const Request& r) {
  return row_tiles(a, r) * a.H * item_steps(a, r);
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
struct Words {
  uint32_t w[kWords];
};

// kWords 32-bit words of the cache, past L1 (every byte is read once).
template <int kWords>
__device__ __forceinline__ void load_words(const int8_t* p, uint32_t* w) {
  if constexpr (kWords == 4) {
    asm("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
        : "l"(p));
  } else if constexpr (kWords == 2) {
    asm("ld.global.nc.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
  } else {
    asm("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
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

// State of one warp for one item: rows r and r + 8 of the tile, r = lane / 4.
template <int D>
struct RowState {
  float acc[D / 8][4];
  float m[2], l[2];  // running maximum (log2 units) and sum of this lane's columns
  float vref;        // power of two at or above the value scales seen
};

// The softmax weights are kept as p * 2^7 * (value scale / vref) in fp16: p is at
// most 2^kSlack (the maximum is moved only when a score passes it by more than
// that), so the largest is 2^15, and weights down to 2^-29 of it keep 11 bits.
constexpr float kSlack = 8.f;
constexpr float kWeightScale = 128.f;

// Rows by 16 keys of one warp.  Q row fragments: lane (r, c), c = lane % 4, holds
// for k-step kk the dims of word kk of the key bytes that the lane itself loads,
// so no byte changes lanes: a key row's chunk of 64 dims is 4 lanes x 16 bytes.
template <int D, typename T, int NQ, int NP>
__global__ void __launch_bounds__(32 * kRowWarps, NQ == 1 && D <= 64 ? 3 : 2) k_kv_rows(AttendArgs a) {
  pdl_enter();
  constexpr int kWK = D >= 64 ? 4 : 2;       // words per load of key bytes
  constexpr int kChunks = D >= 64 ? D / 64 : 1;
  constexpr int kK = kWK * kChunks;          // key words a lane holds per key = MMA k-steps
  constexpr int kWV = D / 32;                // value words a lane holds per key
  constexpr int kRow = D + 4;                // row pitch of the join in shared memory
  __shared__ __align__(16) float s_acc[kRowWarps][kRowTile][kRow];
  __shared__ float s_m[kRowWarps][kRowTile], s_l[kRowWarps][kRowTile], s_v[kRowWarps];
  __shared__ long long s_sum[kRowWarps];
  __shared__ long long s_first[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;

  // ---- this block's share of the steps of all items
  const int per_thread = (a.B + blockDim.x - 1) / blockDim.x;
  const int b_lo = tid * per_thread, b_hi = min(a.B, b_lo + per_thread);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b)
    mine += request_units(a, request_of(a, b, blockIdx.x == 0));
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  __syncthreads();
  long long total = 0;
  for (int i = 0; i < kRowWarps; ++i) {
    if (i < warp) upto += s_sum[i];
    total += s_sum[i];
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < a.min_steps) per = a.min_steps;
  long long u = per * blockIdx.x;
  const long long u_end = min(total, u + per);
  if (u >= u_end) {
    if (tid == 0) a.heads[blockIdx.x].last = -1;
    return;
  }
  if (upto - mine <= u && u < upto) {  // exactly one thread
    long long before = upto - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long x = request_units(a, request_of(a, b, false));
      if (before + x > u) {
        s_first[0] = b;
        s_first[1] = before;
        break;
      }
      before += x;
    }
  }
  __syncthreads();
  int b = (int)s_first[0];
  long long b_units = s_first[1];  // units before request b
  PartHead head = {0, 0, 0, -1};

  while (u < u_end) {
    const Request req = request_of(a, b, false);
    const int64_t tiles = row_tiles(a, req), steps = item_steps(a, req);
    const long long x = tiles * a.H * steps;
    if (b_units + x <= u) {
      b_units += x;
      ++b;
      continue;
    }
    const int64_t item = (u - b_units) / steps;
    const int64_t s0 = (u - b_units) % steps;
    const int64_t s1 = min((long long)steps, s0 + (u_end - u));
    const int h = (int)(item / tiles);
    const int64_t tile = item % tiles;
    const int64_t rows = req.w * a.G;

    // ---- the tile's query rows
    float inv[2];          // score factor of the lane's rows
    int64_t row_hi[2], row_lo[2];
    uint32_t qf[NQ][kK][4];
    const int64_t first_row = tile * kRowTile;
    const int n_rows = (int)min((int64_t)kRowTile, rows - first_row);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t row = first_row + r + 8 * half;
      const bool real = row < rows;
      const int64_t t = real ? row / a.G : 0;
      const T* p = static_cast<const T*>(a.q) + (req.start + t) * a.qsn +
                   (h * a.G + (real ? row % a.G : 0)) * a.qsh;
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
        for (int i = 0; i < 4; ++i) amax = max(amax, __float_as_uint(x[kk][i]) & 0x7FFFFFFFu);
      }
      amax = max(amax, __shfl_xor_sync(kAll, amax, 1));
      amax = max(amax, __shfl_xor_sync(kAll, amax, 2));
      const float f = row_factor(amax);
      inv[half] = __fdiv_rn(a.scale_log2, f);
#pragma unroll
      for (int kk = 0; kk < kK; ++kk) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = f != f ? 0.f : __fmul_rn(x[kk][i], f);
        qf[0][kk][half] = half2_bits(y[0], y[1]);
        qf[0][kk][half + 2] = half2_bits(y[2], y[3]);
        if constexpr (NQ == 2) {
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = __fsub_rn(y[i], __half2float(__float2half_rn(y[i])));
          qf[NQ - 1][kk][half] = half2_bits(y[0], y[1]);
          qf[NQ - 1][kk][half + 2] = half2_bits(y[2], y[3]);
        }
      }
      const int64_t pos = req.L - req.w + t;
      row_hi[half] = real ? (a.causal ? min(req.L, pos + 1) : req.L) : 0;
      row_lo[half] = a.window ? pos - a.window + 1 : 0;
    }
    // keys that any row of the tile sees, and keys that all of them see
    const int64_t t_lo = first_row / a.G, t_hi = (first_row + n_rows - 1) / a.G;
    const int64_t p_lo = req.L - req.w + t_lo, p_hi = req.L - req.w + t_hi;
    const int64_t any_hi = a.causal ? min(req.L, p_hi + 1) : req.L;
    const int64_t any_lo = a.window ? p_lo - a.window + 1 : 0;
    const int64_t all_hi = a.causal ? min(req.L, p_lo + 1) : req.L;
    const int64_t all_lo = a.window ? p_hi - a.window + 1 : 0;
    const int64_t key0 = first_key(a, req) + warp * 16;

    RowState<D> st;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) st.acc[i][0] = st.acc[i][1] = st.acc[i][2] = st.acc[i][3] = 0.f;
    st.m[0] = st.m[1] = -CUDART_INF_F;
    st.l[0] = st.l[1] = 0.f;
    st.vref = 0.f;

    // Block id and scales of step s0 + 32 g + lane, loaded one group ahead.
    int32_t id_n = -1, id_l = -1;
    float ks_n = 0.f, vs_n = 0.f, ks_l = 0.f, vs_l = 0.f;
    auto look_up = [&](int64_t s) {
      const int64_t key = key0 + s * kStepKeys;
      id_n = -1;
      if (s < s1 && key < any_hi && key + 16 > any_lo) {
        id_n = a.table[(int64_t)b * a.max_blocks + (key >> a.bs_log)];
        if (id_n < 0 || id_n >= a.num_blocks) {
          id_n = -1;
          set_status(a.status, kStBadBlock);
        } else {
          ks_n = a.ks[(int64_t)id_n * a.H + h];
          vs_n = a.vs[(int64_t)id_n * a.H + h];
        }
      }
    };
    uint32_t kw[2][2][kK], vw[2][4][kWV];  // [buffer]: key words, value words
    int32_t id_of[2];
    float ks_of[2], vs_of[2];
    auto fetch = [&](int64_t s, int buf) {
      const int at = (int)(s - s0) & 31;
      if (at == 0) {
        id_l = id_n;
        ks_l = ks_n;
        vs_l = vs_n;
        look_up(s + 32 + lane);
      }
      const int32_t id = s < s1 ? __shfl_sync(kAll, id_l, at) : -1;
      id_of[buf] = id;
      ks_of[buf] = __shfl_sync(kAll, ks_l, at);
      vs_of[buf] = __shfl_sync(kAll, vs_l, at);
      if (id < 0) return;
      const int64_t key = key0 + s * kStepKeys;
      const int64_t off = ((((int64_t)id * a.H + h) << a.bs_log) + (key & ((1 << a.bs_log) - 1))) * D;
      const int8_t* kp = a.k + off + r * D + c * (4 * kWK);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          load_words<kWK>(kp + j * 8 * D + i * 64, &kw[buf][j][i * kWK]);
      const int8_t* vp = a.v + off + 2 * c * D + r * (D / 8);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        load_words<kWV>(vp + ((j & 1) + (j >> 1) * 8) * D, vw[buf][j]);
    };
    auto compute = [&](int64_t s, int buf) {
      if (id_of[buf] < 0) return;
      const int64_t key = key0 + s * kStepKeys;
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int kk = 0; kk < kK; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = kw[buf][j][kk] ^ 0x80808080u;
          const uint32_t b0 = codes_half2(x, kSelLow), b1 = codes_half2(x, kSelHigh);
          mma_16816(sc[j], qf[0][kk], b0, b1);
          if constexpr (NQ == 2) mma_16816(sc[j], qf[NQ - 1][kk], b0, b1);
        }
      const float ks = isfinite(ks_of[buf]) ? ks_of[buf] : CUDART_NAN_F;
      const float vs = vs_of[buf];
      const float f[2] = {__fmul_rn(inv[0], ks), __fmul_rn(inv[1], ks)};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[j][i] = __fmul_rn(sc[j][i], f[i >> 1]);
      if (key + 16 > all_hi || key < all_lo) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t at = key + j * 8 + 2 * c + (i & 1);
            if (at >= row_hi[i >> 1] || at < row_lo[i >> 1]) sc[j][i] = -CUDART_INF_F;
          }
      }
      const float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      const float mx1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
      const float va = fabsf(vs);
      const bool vup = va > st.vref && va < CUDART_INF_F;
      if (__any_sync(kAll, mx0 > st.m[0] + kSlack || mx1 > st.m[1] + kSlack || vup)) {
        float beta = 1.f;
        if (vup) {  // the next power of two
          const uint32_t e = (__float_as_uint(va) >> 23) + 1;
          const float to = __uint_as_float((e > 254 ? 254 : e) << 23);
          beta = __fdiv_rn(st.vref, to);
          st.vref = to;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float mx = half ? mx1 : mx0;
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
          const float to = fmaxf(st.m[half], mx);
          const float alpha = to == st.m[half] ? 1.f : exp2_fast(st.m[half] - to);
          st.m[half] = to;
          st.l[half] = __fmul_rn(st.l[half], alpha);
          const float g = __fmul_rn(alpha, beta);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            st.acc[i][2 * half] = __fmul_rn(st.acc[i][2 * half], g);
            st.acc[i][2 * half + 1] = __fmul_rn(st.acc[i][2 * half + 1], g);
          }
        }
      }
      const float pv = isfinite(vs) ? (st.vref > 0.f ? __fmul_rn(__fdiv_rn(vs, st.vref), kWeightScale) : 0.f)
                                    : CUDART_NAN_F;
      float p[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = st.m[i >> 1];
          const float e = exp2_fast(__fsub_rn(sc[j][i], m == -CUDART_INF_F ? 0.f : m));
          st.l[i >> 1] = __fadd_rn(st.l[i >> 1], e);
          // a hidden key has weight 0 whatever its block's scale is
          p[j][i] = sc[j][i] == -CUDART_INF_F ? 0.f : __fmul_rn(e, pv);
        }
      uint32_t pa[NP][4];
#pragma unroll
      for (int t = 0; t < NP; ++t) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            pa[t][2 * j + half] = half2_bits(p[j][2 * half], p[j][2 * half + 1]);
        if (t + 1 < NP) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              p[j][i] = __fsub_rn(p[j][i], __half2float(__float2half_rn(p[j][i])));
        }
      }
#pragma unroll
      for (int w = 0; w < kWV; ++w) {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = vw[buf][j][w] ^ 0x80808080u;
        const uint32_t lo0 = __byte_perm(x[0], x[1], 0x5140), hi0 = __byte_perm(x[0], x[1], 0x7362);
        const uint32_t lo1 = __byte_perm(x[2], x[3], 0x5140), hi1 = __byte_perm(x[2], x[3], 0x7362);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sel = e & 1 ? kSelHigh : kSelLow;
          const uint32_t b0 = codes_half2(e < 2 ? lo0 : hi0, sel);
          const uint32_t b1 = codes_half2(e < 2 ? lo1 : hi1, sel);
          mma_16816(st.acc[w * 4 + e], pa[0], b0, b1);
          if constexpr (NP == 2) mma_16816(st.acc[w * 4 + e], pa[NP - 1], b0, b1);
        }
      }
    };

    look_up(s0 + lane);
    fetch(s0, 0);
    for (int64_t s = s0; s < s1; s += 2) {
      fetch(s + 1, 1);
      compute(s, 0);
      fetch(s + 2, 0);
      if (s + 1 < s1) compute(s + 1, 1);
    }

    // ---- the warps' parts of the item together
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      st.l[half] += __shfl_xor_sync(kAll, st.l[half], 1);
      st.l[half] += __shfl_xor_sync(kAll, st.l[half], 2);
      if (r + 8 * half < n_rows) {
        float* to = &s_acc[warp][r + 8 * half][2 * c * (D / 8)];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < D / 8; i += 4)
            *reinterpret_cast<float4*>(to + j * (D / 8) + i) =
                make_float4(st.acc[i][2 * half + j], st.acc[i + 1][2 * half + j],
                            st.acc[i + 2][2 * half + j], st.acc[i + 3][2 * half + j]);
      }
      if (c == 0) {
        s_m[warp][r + 8 * half] = st.m[half];
        s_l[warp][r + 8 * half] = st.l[half];
      }
    }
    if (lane == 0) s_v[warp] = __fmul_rn(st.vref, 1.f / kWeightScale);
    __syncthreads();
    const bool begins = s0 == 0, ends = s1 == steps;
    float* part = a.parts + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kRowTile * (D + 2);
    for (int i = tid; i < n_rows * (D / 4); i += blockDim.x) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float M = s_m[0][row], L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 1; w < kRowWarps; ++w) M = fmaxf(M, s_m[w][row]);
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        const float l = s_l[w][row], m = s_m[w][row];
        if (l == 0.f) continue;  // this warp saw no key of the row
        const float e = m == -CUDART_INF_F ? 1.f : exp2_fast(m - M);
        const float g = __fmul_rn(e, s_v[w]);
        L = __fmaf_rn(l, e, L);
        const float4 v = *reinterpret_cast<const float4*>(&s_acc[w][row][d]);
        o[0] = __fmaf_rn(v.x, g, o[0]);
        o[1] = __fmaf_rn(v.y, g, o[1]);
        o[2] = __fmaf_rn(v.z, g, o[2]);
        o[3] = __fmaf_rn(v.w, g, o[3]);
      }
      if (begins && ends) {
        const int64_t at = first_row + row, t = at / a.G;
        const int hq = h * a.G + (int)(at % a.G);
        const float g = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = L == 0.f ? 0.f : __fmul_rn(o[j], g);
        store4<T>(static_cast<T*>(a.out) + (req.start + t) * a.osn + hq * a.osh + d, o);
        if (a.lse && d == 0)
          a.lse[(req.start + t) * a.Hq + hq] =
              L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
      } else {
        *reinterpret_cast<float2*>(part + row * (D + 2) + d) = make_float2(o[0], o[1]);
        *reinterpret_cast<float2*>(part + row * (D + 2) + d + 2) = make_float2(o[2], o[3]);
        if (d == 0) *reinterpret_cast<float2*>(part + row * (D + 2) + D) = make_float2(M, L);
      }
    }
    if (begins && !ends) {
      head.b = b;
      head.h = h;
      head.tile = (int)tile;
      head.last = (int)((b_units + (item + 1) * steps - 1) / per);
    }
    u += s1 - s0;
    __syncthreads();
  }
  if (tid == 0) a.heads[blockIdx.x] = head;
}

// Joins the parts of the items that k_kv_rows split: block i takes the item that
// begins in block i there and goes on into the next ones.
template <int D, typename T>
__global__ void __launch_bounds__(256) k_kv_join(AttendArgs a) {
  pdl_enter();
  const PartHead head = a.heads[blockIdx.x];
  if (head.last < 0) return;
  const Request req = request_of(a, head.b, false);
  const int64_t first_row = (int64_t)head.tile * kRowTile, rows = req.w * a.G;
  const int n_rows = (int)min((int64_t)kRowTile, rows - first_row);
  const int first = blockIdx.x;
  constexpr int64_t kPart = (int64_t)kRowTile * (D + 2);
  auto part = [&](int i) { return a.parts + ((int64_t)i * 2 + (i == first ? 1 : 0)) * kPart; };
  for (int i = threadIdx.x; i < n_rows * (D / 4); i += blockDim.x) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    float M = -CUDART_INF_F, L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = first; j <= head.last; ++j) M = fmaxf(M, part(j)[row * (D + 2) + D]);
    for (int j = first; j <= head.last; ++j) {
      const float* p = part(j) + row * (D + 2);
      const float m = p[D], l = p[D + 1];
      if (l == 0.f) continue;
      const float e = m == -CUDART_INF_F ? 1.f : exp2_fast(m - M);
      L = __fmaf_rn(l, e, L);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __fmaf_rn(p[d + k], e, o[k]);
    }
    const int64_t at = first_row + row, t = at / a.G;
    const int hq = head.h * a.G + (int)(at % a.G);
    const float g = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = L == 0.f ? 0.f : __fmul_rn(o[j], g);
    store4<T>(static_cast<T*>(a.out) + (req.start + t) * a.osn + hq * a.osh + d, o);
    if (a.lse && d == 0)
      a.lse[(req.start + t) * a.Hq + hq] =
          L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
  }
}

}  // namespace mpzch_kv
