// Element access and elementwise functions shared by the layers beside the memory: convolution, scan, linear attention,
// norms and projections.
#pragma once

#include <cuda_bf16.h>

#include "sdm_internal.cuh"

namespace sdm {

// A 16-byte piece of a row: 8 bf16 or 4 fp32 elements.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  static constexpr int n = 4;
  __device__ static void load(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  __device__ static uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void load(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of an fp32
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ static uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float* p) { *p = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {  // at most 2 units in the last place
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest float for infinity: a factor that times a state of 0 is 0.  NaN stays.
__device__ __forceinline__ float at_most_finite(float x) { return x > 3.402823466e38f ? 3.402823466e38f : x; }

__device__ __forceinline__ float rcp_fast(float x) {  // one unit in the last place; 0 for inf
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-x).  For x below about -88 the exponential is inf and the result 0.
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_fast(1.0f + exp2_fast(-kLog2e * x));
}
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1], of two values.  log(1 + e) = e p(e)
// keeps its relative precision where e is tiny (the logarithm of the rounded 1 + e would not), so a
// step size of 1e-3 is as exact as one of 1.  p is the polynomial of degree 8 nearest to
// log(1 + e) / e on [0, 1] in relative error (3e-8; 2e-7 with its roundings), by weighted least
// squares on Chebyshev points, the weights moved until the error was level.
__device__ __forceinline__ uint64_t softplus2(uint64_t x) {
  float x0, x1;
  unpack2(x, x0, x1);
  const uint64_t e = pack2(exp2_fast(-kLog2e * fabsf(x0)), exp2_fast(-kLog2e * fabsf(x1)));
  auto both = [](float v) { return pack2(v, v); };
  uint64_t p = fma2(e, both(0.0052326880395412445f), both(-0.029505213722586632f));
  p = fma2(e, p, both(0.07822591066360474f));
  p = fma2(e, p, both(-0.13663242757320404f));
  p = fma2(e, p, both(0.19106005132198334f));
  p = fma2(e, p, both(-0.2484298199415207f));
  p = fma2(e, p, both(0.3331909775733948f));
  p = fma2(e, p, both(-0.4999949336051941f));
  p = fma2(e, p, both(0.9999999403953552f));
  return fma2(e, p, pack2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
}
__device__ __forceinline__ float softplus(float x) {
  float a, b;
  unpack2(softplus2(pack2(x, x)), a, b);
  return a;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory, zeros where !in.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
// One element where rows are not aligned to 16 bytes: 4 bytes are copied like 16, 2 bytes are loaded.
__device__ __forceinline__ void copy1(float* dst, const float* src, bool in) {
  const int n = in ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy1(__nv_bfloat16* dst, const __nv_bfloat16* src, bool in) {
  *dst = in ? *src : __nv_bfloat16(0.f);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// A state carried over a chunk that adds `end` to it: exp(sum A) h + end.  Where the state grows, the
// factor may pass the largest float although its product with h, and each token's own factor, do
// not: it is then applied in two halves, and a state of 0 stays 0.
__device__ __forceinline__ float carried_up(float h, float sum, float rate, float end) {
  const float e = fmaf(sum, rate, 2.0e-8f);
  if (!(e > 64.0f)) return fmaf(exp2_fast(e), h, end);
  const float half = exp2_fast(0.5f * e);
  return h == 0.0f ? end : fmaf(half, half * h, end);
}

// The memory of a tensor of a call: n1 x n2 rows of `bytes`, s1 and s2 bytes apart.
struct Extent {
  const void* p;
  long long n1, s1, n2, s2, bytes;
};
inline Extent dense(const void* p, long long bytes) { return {p, 1, 0, 1, 0, bytes}; }

// Whether any byte of `e` lies in the `bytes` from p on.
inline bool meets(const Extent& e, const void* p, long long bytes) {
  if (!e.p || !p || e.n1 < 1 || e.n2 < 1 || e.bytes < 1 || bytes < 1) return false;
  // a: the start of e's lowest row, as a distance from p
  long long a = (long long)(reinterpret_cast<uintptr_t>(e.p) - reinterpret_cast<uintptr_t>(p));
  long long n1 = e.n1, n2 = e.n2, s1 = e.s1, s2 = e.s2;
  if (s1 < 0) a += (n1 - 1) * s1, s1 = -s1;
  if (s2 < 0) a += (n2 - 1) * s2, s2 = -s2;
  if (a >= bytes || a + (n1 - 1) * s1 + (n2 - 1) * s2 + e.bytes <= 0) return false;
  if (n1 > n2) {
    long long t = n1;
    n1 = n2, n2 = t;
    t = s1, s1 = s2, s2 = t;
  }
  // Row by row of the shorter direction: the first row of the other that ends past p starts before
  // the end, or none does.
  for (long long i = 0; i < n1; ++i, a += s1) {
    const long long short_by = -(a + e.bytes);  // 0 or more: row 0 ends before p
    const long long j = short_by < 0 ? 0 : s2 ? short_by / s2 + 1 : n2;
    if (j < n2 && a + j * s2 < bytes) return true;
  }
  return false;
}

// The sequence length of batch row b, clamped to [0, T] (T without lengths).
__device__ __forceinline__ int row_length(const int32_t* lengths, int b, int T) {
  return lengths ? min(max(lengths[b], 0), T) : T;
}

// The state row of batch row b: its slot, or -1 for a padding row.  A slot past the pool is
// reported and treated as padding, so no access leaves the pool.  Asked for first and looked at
// later (checked_slot), it is on its way while everything that does not need it is asked for too.
__device__ __forceinline__ int asked_slot(const int32_t* slots, int b) { return slots ? slots[b] : b; }
__device__ __forceinline__ int checked_slot(const int32_t* slots, int slot, int n_slots, int* dev_err) {
  if (!slots || slot < n_slots) return slot < 0 ? -1 : slot;
  if (dev_err) atomicOr(dev_err, SDM_DEV_INDEX_RANGE);
  return -1;
}
__device__ __forceinline__ int row_slot(const int32_t* slots, int b, int n_slots, int* dev_err) {
  return checked_slot(slots, asked_slot(slots, b), n_slots, dev_err);
}

}  // namespace sdm
