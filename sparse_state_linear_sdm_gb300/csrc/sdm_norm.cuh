// What the norms and their gradient share (sdm_norm.cu, sdm_norm_backward.cu): rows in registers, sums over a row.
#pragma once

#include "sdm_layers.cuh"

namespace sdm {

constexpr int kNormMax = 16384;  // channels of a row (of a group)

// A row of n channels held by TPR threads, E = 8 P channels each.  VEC: in pieces of eight, which are 16-byte words
// of bf16 and pairs of them of fp32; otherwise (rows off 16 bytes, n not a multiple of 8) one by one in turn, so that a warp's
// accesses are consecutive either way.
template <int TPR, int P, bool VEC>
struct Row {
  static constexpr int E = 8 * P;
  // The channel of this thread's element e.
  __device__ static int at(int t, int e) { return VEC ? (e / 8 * TPR + t) * 8 + e % 8 : e * TPR + t; }

  template <typename T>
  __device__ static void load(const T* p, int t, int n, float (&v)[E]) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = (i * TPR + t) * 8;
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int k = 0; k < int(sizeof(T)) / 2; ++k)
          w[k] = c < n ? *(reinterpret_cast<const uint4*>(p + c) + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < int(sizeof(T)) / 2; ++k) {
          float f[Piece<T>::n];
          Piece<T>::load(w[k], f);
#pragma unroll
          for (int j = 0; j < Piece<T>::n; ++j) v[8 * i + k * Piece<T>::n + j] = f[j];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = at(t, e) < n ? to_f32(p[at(t, e)]) : 0.f;
    }
  }
  template <typename T>
  __device__ static void store(T* p, int t, int n, const float (&v)[E]) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = (i * TPR + t) * 8;
        if (c >= n) break;
#pragma unroll
        for (int k = 0; k < int(sizeof(T)) / 2; ++k) {
          float f[Piece<T>::n];
#pragma unroll
          for (int j = 0; j < Piece<T>::n; ++j) f[j] = v[8 * i + k * Piece<T>::n + j];
          *(reinterpret_cast<uint4*>(p + c) + k) = Piece<T>::pack(f);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (at(t, e) < n) from_f32(v[e], p + at(t, e));
    }
  }
  // A weight vector of either type from channel `off` on.
  __device__ static void weights(const void* p, int dtype, long long off, int t, int n, float (&v)[E]) {
    if (dtype == SDM_F32)
      load(static_cast<const float*>(p) + off, t, n, v);
    else
      load(static_cast<const __nv_bfloat16*>(p) + off, t, n, v);
  }
};

// Sums of K values over the TPR threads of a row; every thread of the block calls it.  `part` is this call's own.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&v)[K], float (*part)[K]) {
#pragma unroll
  for (int m = (TPR < 32 ? TPR : 32) / 2; m > 0; m /= 2)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], m);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int w = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[w][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += part[i][k];
      v[k] = s;
    }
  }
}

constexpr int norm_block(int tpr) { return tpr < 128 ? 128 : tpr; }

// The instances: threads of a row and pieces of a thread by the row's channels.
template <template <typename, typename, int, int, bool> class Launch, typename TX, typename TR, bool VEC, typename... A>
int norm_by_width(int n, A&&... a) {
  if (n <= 64) return Launch<TX, TR, 8, 1, VEC>::run(a...);
  if (n <= 128) return Launch<TX, TR, 16, 1, VEC>::run(a...);
  if (n <= 256) return Launch<TX, TR, 32, 1, VEC>::run(a...);
  if (n <= 1024) return Launch<TX, TR, 64, 2, VEC>::run(a...);
  if (n <= 2048) return Launch<TX, TR, 128, 2, VEC>::run(a...);
  if (n <= 4096) return Launch<TX, TR, 256, 2, VEC>::run(a...);
  if (n <= 8192) return Launch<TX, TR, 512, 2, VEC>::run(a...);
  return Launch<TX, TR, 512, 4, VEC>::run(a...);
}
template <template <typename, typename, int, int, bool> class Launch, typename... A>
int norm_dispatch(int x_dtype, int r_dtype, bool vec, int n, A&&... a) {
  typedef __nv_bfloat16 H;
  if (x_dtype == SDM_F32)
    return vec ? norm_by_width<Launch, float, float, true>(n, a...) : norm_by_width<Launch, float, float, false>(n, a...);
  if (r_dtype == SDM_F32)
    return vec ? norm_by_width<Launch, H, float, true>(n, a...) : norm_by_width<Launch, H, float, false>(n, a...);
  return vec ? norm_by_width<Launch, H, H, true>(n, a...) : norm_by_width<Launch, H, H, false>(n, a...);
}

inline uintptr_t norm_odd(int dtype) { return dtype == SDM_F32 ? 3 : 1; }
inline bool misaligned(const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; }

// Checks that both directions share.
inline int check_norm(const sdm_norm_args& a) {
  if (a.M < 0 || a.D < 1 || a.groups < 1 || a.D % a.groups || bad_dtype(a.x_dtype) || bad_dtype(a.r_dtype) ||
      bad_dtype(a.w_dtype) || !(a.eps >= 0.f))
    return SDM_EINVAL;
  if (a.act != SDM_ACT_NONE && a.act != SDM_ACT_SILU) return SDM_EINVAL;
  if (a.weight && a.groups > 1) return SDM_EINVAL;            // the second norm is over whole rows
  if (a.x_dtype == SDM_F32 && a.r_dtype != SDM_F32) return SDM_EUNSUPPORTED;
  if (a.D / a.groups > kNormMax || a.M > 0x7FFFFFFFLL / a.groups) return SDM_EUNSUPPORTED;
  const uintptr_t w = norm_odd(a.w_dtype);
  if (misaligned(a.after, w) || misaligned(a.scale, w) || misaligned(a.weight, w)) return SDM_EALIGN;
  return SDM_OK;
}
inline int norm_es(int dtype) { return dtype == SDM_F32 ? 4 : 2; }
inline Extent norm_rows(const void* p, long long M, long long rs, int D, int es) {
  return Extent{p, M, rs * es, 1, 0, (long long)D * es};
}
// Whether e's rows are where the dense rows at p lie: a thread then writes what only it has read.
inline bool same_rows(const Extent& e, const void* p, long long row_bytes) {
  return e.p == p && e.bytes == row_bytes && (e.n1 == 1 || e.s1 == row_bytes);
}

}  // namespace sdm
