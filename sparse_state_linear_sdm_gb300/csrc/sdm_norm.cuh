// What the norms and their gradient share (sdm_norm.cu, sdm_norm_backward.cu): rows in registers, sums over a row.
#pragma once

#include <type_traits>

#include "sdm_layers.cuh"

namespace sdm {

constexpr int kNormMax = 16384;  // channels of a row (of a group)

// A row of n channels held by TPR threads, E = 8 P channels each.  VEC: in pieces of eight, which are 16-byte words
// of bf16 and pairs of them of fp32; otherwise (rows off 16 bytes, n not a multiple of 8) one by one in turn, so that a warp's
// accesses are consecutive either way.
template <int TPR, int P, bool VEC, bool SURE = true>
struct Row {
  static constexpr int E = 8 * P;
  // The channel of this thread's element e.
  __device__ static int at(int t, int e) { return VEC ? (e / 8 * TPR + t) * 8 + e % 8 : e * TPR + t; }
  // A block's only row; it always has channels.  Of several, those past the last row have none.
  static constexpr bool kAlone = TPR >= 128;
  // One by one: whether element e of a row that has channels is inside.  But for the shortest rows the first half is, which
  // SURE takes for granted (the stream's gradient, 16384 x 2047: 81 us without, 75).
  __device__ static bool inside(int t, int e, int n) { return (SURE && TPR > 8 && e < E / 2) || at(t, e) < n; }

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
      if (!kAlone && n == 0) return;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (inside(t, e, n)) from_f32(v[e], p + at(t, e));
    }
  }
  // The same in two steps: asked for, and later taken as numbers.
  template <typename T>
  struct Raw {
    static constexpr int N = VEC ? P * int(sizeof(T)) / 2 : 1;
    uint4 w[N];
    T v[VEC ? 1 : E];
    __device__ void ask(const T* p, int t, int n) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = (i * TPR + t) * 8;
#pragma unroll
          for (int k = 0; k < int(sizeof(T)) / 2; ++k)
            w[i * (int(sizeof(T)) / 2) + k] = c < n ? *(reinterpret_cast<const uint4*>(p + c) + k) : make_uint4(0, 0, 0, 0);
        }
      } else {
        if (!kAlone && n == 0) {
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = T(0.f);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = inside(t, e, n) ? p[at(t, e)] : T(0.f);
        }
      }
    }
    __device__ void get(float (&f)[E]) const {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float x[Piece<T>::n];
          Piece<T>::load(w[i], x);
#pragma unroll
          for (int j = 0; j < Piece<T>::n; ++j) f[i * Piece<T>::n + j] = x[j];
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = to_f32(v[e]);
      }
    }
  };
  // A weight vector of either type from channel `off` on.
  __device__ static void weights(const void* p, int dtype, long long off, int t, int n, float (&v)[E]) {
    if (dtype == SDM_F32)
      load(static_cast<const float*>(p) + off, t, n, v);
    else
      load(static_cast<const __nv_bfloat16*>(p) + off, t, n, v);
  }
};

// Sum of N warps' parts, in log2 N roundings.
template <int N, int K>
__device__ __forceinline__ float tree_sum(const float (*part)[K], int k) {
  if constexpr (N == 1)
    return part[0][k];
  else
    return tree_sum<N / 2, K>(part, k) + tree_sum<N / 2, K>(part + N / 2, k);
}
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
    for (int k = 0; k < K; ++k) v[k] = tree_sum<W, K>(part + w / W * W, k);  // the row's own warps
  }
}

constexpr int norm_block(int tpr) { return tpr < 128 ? 128 : tpr; }

// Threads of a row and pieces of a thread by the row's channels, calling f(threads, pieces): eight channels a thread up to
// 4096, then as many more as a block of at most `most` threads leaves.
template <int MOST, bool TWO = false, typename F>
auto norm_by_width(int n, F f) {
  typedef std::integral_constant<int, 1> One;
  if (n <= 64) return f(std::integral_constant<int, 8>(), One());
  if (n <= 128) return f(std::integral_constant<int, 16>(), One());
  if (n <= 256) return f(std::integral_constant<int, 32>(), One());
  if (n <= 512) return f(std::integral_constant<int, 64>(), One());
  if (n <= 1024) return f(std::integral_constant<int, 128>(), One());
  if (n <= 2048) return f(std::integral_constant<int, 256>(), One());
  if (TWO && n <= 4096) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  if (n <= 4096) return f(std::integral_constant<int, 512>(), One());
  if (n <= 8192) return f(std::integral_constant<int, MOST>(), std::integral_constant<int, 1024 / MOST>());
  return f(std::integral_constant<int, MOST>(), std::integral_constant<int, 2048 / MOST>());
}

// A thread's own copies of the weights in shared memory: asked for row by row they waited for L2 behind the rows that
// pass through L1.
template <typename R, int BLOCK, int N>
struct Kept {
  static constexpr bool on = R::E == 8;
  float4 v[on ? N * 2 * BLOCK : 1];
  __device__ void put(int which, const void* p, int dtype, long long off, int t, int n) {
    if constexpr (on) {
      float w[R::E];
      R::weights(p, dtype, off, t, n, w);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        v[(which * 2 + k) * BLOCK + threadIdx.x] = make_float4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    }
  }
  __device__ void get(int which, const void* p, int dtype, long long off, int t, int n, float (&w)[R::E]) const {
    if constexpr (on) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 x = v[(which * 2 + k) * BLOCK + threadIdx.x];
        w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
      }
    } else {
      R::weights(p, dtype, off, t, n, w);
    }
  }
};

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
