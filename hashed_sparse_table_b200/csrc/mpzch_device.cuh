// Device helpers shared by the table kernels and the history-cache kernels:
// status bits, programmatic dependent launch, the clock of bounded waits and the
// int8 rounding of the export.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace mpzch {

__device__ __forceinline__ void set_status(int32_t* st, int bits) {
  if (st) atomicOr(st, bits);
}

// Waits on other warps or on copies in flight give up after this long and set
// MPZCH_STATUS_TIMEOUT (far beyond any legitimate wait).
constexpr int kStTimeout = 16;
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Programmatic dependent launch.  pdl_enter waits until every earlier grid of
// the stream has completed and its memory is visible; every kernel calls it
// first, so nothing is read before the producer has finished.  pdl_trigger
// lets the next kernel of the stream launch; kernels of the row-map chain call
// it once their main work is done, so the next kernel's blocks are scheduled
// during this kernel's tail rather than parked on the SMs (holding warps and
// shared memory that the concurrently running row kernels need) for its whole
// run.  A kernel that never calls it triggers when its blocks exit.  Both are
// no-ops for a kernel launched without the programmatic-serialisation
// attribute.
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void pdl_enter() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Round-half-to-even of |v| < 2^22 without a conversion instruction: adding
// 1.5 * 2^23 leaves v's nearest integer (ties to even, IEEE rounding of the
// add) in the low mantissa bits, and subtracting it again gives that integer as
// a float.  Only full-rate FP32 / integer operations.
constexpr float kRoundMagic = 12582912.0f;  // 1.5 * 2^23
constexpr int kRoundMagicBits = 0x4B400000;

__device__ __forceinline__ int rne_small(float v) {
  return __float_as_int(__fadd_rn(v, kRoundMagic)) - kRoundMagicBits;
}

// int8 export rule, q = rne(fl(x / s)) clamped to +-127, for the values of one
// lane.  p = fl(x * fl(1/s)) differs from the exact quotient t = x/s by at most
// |t| 2^-23 + |t| 2^-24, and fl(t) from t by at most |t| 2^-24, so
// |p - fl(x/s)| < |t| 2^-22 <= 127.00001 * 2^-22 < 3.1e-5.  When p is more than
// 1e-4 away from every half-integer, fl(x/s) rounds to the same integer as p; a
// lane with any value closer than that (or with no usable reciprocal, for a
// subnormal s) recomputes all of its values from the IEEE quotient.
// |x| <= a = 127 s, so every code lies in [-127, 127] (clamped all the same).
template <int kN>
__device__ __forceinline__ void quant_lane(const float (&x)[kN], float s, float rcp, bool fast,
                                           int (&t)[kN]) {
  bool amb = !fast;
#pragma unroll
  for (int e = 0; e < kN; ++e) {
    const float p = __fmul_rn(x[e], rcp);
    const float y = __fadd_rn(p, kRoundMagic);
    const float r = __fsub_rn(y, kRoundMagic);
    amb |= fabsf(__fsub_rn(p, r)) > 0.4999f;
    t[e] = __float_as_int(y) - kRoundMagicBits;
  }
  if (amb) {
#pragma unroll
    for (int e = 0; e < kN; ++e) t[e] = rne_small(__fdiv_rn(x[e], s));
  }
#pragma unroll
  for (int e = 0; e < kN; ++e) t[e] = max(-127, min(127, t[e]));
}

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

}  // namespace mpzch
