// Projections with bias, activation and residual, and their gradient, on the tcgen05 tensor cores (sdm_product.cuh).
//
//   z = x w^T + bias,   y = residual + act(z)                      (w [N, D])
//   dz = dy act'(z),    dx = dz w,   dw = dz^T x,   dbias = sum of dz over tokens
//
// Sums are fp32 and y is rounded once.  dz is rounded to bf16 between the products (as the gated projections' dg and
// du: the tensor cores take nothing wider at that rate), and dbias sums the rounded values; without an activation dz is dy itself.
//
// 16,384 tokens of 8192 x 2048 with a residual: 350 to 356 us by GPU, 1,545 to 1,570 TFLOP/s (0.81 of cuBLAS's burst, 0.91
// of its sustained rate).  The gradient of 1000 tokens of 1024 x 2736 with gelu: 39 us, its slope pass 44 tiles on 76 pairs.  4 tokens of
// 8192 x 2048: 9.6 (0.52 of the HBM floor), of which a launch is 3 to 4.
#include "sdm_product.cuh"

namespace sdm {
namespace {

// ---- few tokens ----
//
// HBM bounds a decode step's product: all of w for a handful of tokens.  A block takes 16 rows of w, the rows of one
// mma.m16n8k16 with tokens as its columns, in 16-byte words straight from global memory as sdm_gated.cu's kernel does.
// Where N is short of blocks a block has more warps for its reduction; their sums meet in shared memory in their order.
constexpr int kFewRows = 16;

template <int ACT, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) few_dense_kernel(const __nv_bfloat16* __restrict__ x,
                                                               const __nv_bfloat16* __restrict__ w,
                                                               const __nv_bfloat16* __restrict__ bias,
                                                               const __nv_bfloat16* residual, int M, int D, int N,
                                                               __nv_bfloat16* y) {
  constexpr int kAhead = 8 / NT;
  __shared__ float4 part[WARPS][NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int n0 = int(blockIdx.x) * kFewRows + g;
  const bool second = n0 + 8 < N;  // N % 8 == 0: the first row is always inside
  const __nv_bfloat16* wa = w + size_t(n0) * D + c * 8;
  const __nv_bfloat16* wb = wa + size_t(8) * D;
  const __nv_bfloat16* xr = x + size_t(g) * D + c * 8;

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * 32 * kAhead; k0 < D; k0 += WARPS * 32 * kAhead) {
    uint4 va[kAhead], vb[kAhead], vx[kAhead][NT];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j * 32;
      const bool in = k + c * 8 < D;  // D % 8 == 0
      va[j] = in ? load_stream(wa + k) : zero;
      vb[j] = in && second ? load_stream(wb + k) : zero;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        vx[j][t] = in && t * 8 + g < M ? *reinterpret_cast<const uint4*>(xr + size_t(t) * 8 * D + k) : zero;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16n8(acc[t], va[j].x, vb[j].x, va[j].y, vb[j].y, vx[j][t].x, vx[j][t].y);
        mma16n8(acc[t], va[j].z, vb[j].z, va[j].w, vb[j].w, vx[j][t].z, vx[j][t].w);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) part[warp][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  __syncthreads();
  if (warp < NT) {  // row n0 of tokens m, m + 1 in x, y; row n0 + 8 in z, w
    float4 s = part[0][warp][lane];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) {
      const float4 p = part[i][warp][lane];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    const int m = warp * 8 + 2 * c;
    const float z[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = n0 + (i / 2) * 8, tok = m + i % 2;
      if (tok >= M || (i >= 2 && !second)) continue;
      const size_t at = size_t(tok) * N + row;
      float v = dense_act<ACT>(z[i] + (bias ? __bfloat162float(bias[row]) : 0.f));
      if (residual) v += __bfloat162float(residual[at]);
      y[at] = __float2bfloat16_rn(v);
    }
  }
}

template <int ACT, int NT, int WARPS>
int launch_few_dense(const void* x, const void* w, const void* bias, const void* residual, int M, int D, int N, void* y,
                     cudaStream_t s) {
  typedef const __nv_bfloat16* P;
  few_dense_kernel<ACT, NT, WARPS><<<unsigned(ceil_div(N, kFewRows)), WARPS * 32, 0, s>>>(
      static_cast<P>(x), static_cast<P>(w), static_cast<P>(bias), static_cast<P>(residual), M, D, N,
      static_cast<__nv_bfloat16*>(y));
  return last_launch_status();
}
// Warps of a block: enough of them on the card where its blocks are few and their reductions long.  4 tokens of 8192 x 2048 take
// 11.7 us with 4 warps, 8.8 with 8 and 8.2 with 16, of 4096 x 4096 8.8, 7.8 and 9.8, of 2048 x 2048 3.9, 3.3 and 3.4; 8 of
// 2048 x 8192 8.0, 9.4 and 12.7.  (The reduction over a cluster's CTAs took 8.9, 9.5, 4.2 and 7.7.)
template <int ACT, int NT>
int launch_few_dense(const void* x, const void* w, const void* bias, const void* residual, int M, int D, int N, void* y,
                     cudaStream_t s) {
  const int blocks = ceil_div(N, kFewRows);
  if (blocks <= 128 && D >= 4096) return launch_few_dense<ACT, NT, 16>(x, w, bias, residual, M, D, N, y, s);
  if (blocks <= 256 && D >= 2048) return launch_few_dense<ACT, NT, 8>(x, w, bias, residual, M, D, N, y, s);
  return launch_few_dense<ACT, NT, 4>(x, w, bias, residual, M, D, N, y, s);
}
template <int ACT>
int launch_few_act(const void* x, const void* w, const void* bias, const void* residual, int M, int D, int N, void* y,
                   cudaStream_t s) {
  return M <= 8 ? launch_few_dense<ACT, 1>(x, w, bias, residual, M, D, N, y, s)
                : launch_few_dense<ACT, 2>(x, w, bias, residual, M, D, N, y, s);
}

// ---- the tiles ----

// A product by itself, its reduction split where its tiles leave pairs of SMs idle: the cut of least time.
Product plan_dense(int M, int D, int N) {
  // Row tiles of a group: with a short reduction the outputs weigh more (16,384 tokens of 2048 x 2048: 101 us in groups
  // of 4, 111 of 16), with a long one the rows of x that are read again (8192 x 2048: 330 us and 303, 320 of 32).
  Product p = product(M, N, 2 * kHalf, D);
  p.group = D <= 2048 ? 4 : 16;
  if ((long long)p.row_tiles * p.col_tiles >= 2 * kPairs) return p;
  Product best = p;
  const Product none = {};
  double least = -1;
  for (int i = 1; i <= 32; ++i) {
    cut(p, i);
    const double t = busiest(p, none) + joining(p);
    if (least < 0 || t < least) {
      least = t;
      best = p;
    }
  }
  return best;
}

template <int MODE, int ACT>
int launch_dense_act(const Maps& tm, const ProductArgs& a, cudaStream_t s) {
  const int st = launch_mode<MODE, ACT>(tm, a, s);
  if (st != SDM_OK || a.p[0].splits == 1) return st;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((size_t(a.p[0].rows) * a.p[0].cols / 8 + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_dense_kernel<MODE, ACT>, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}
// MODE's product of x and w with its epilogue into out.
template <int MODE>
int launch_dense(const void* x, const void* w, const void* bias, const void* extra, int M, int D, int N, int act, void* out,
                 void* partial, float* sums, int* dev_err, cudaStream_t s) {
  ProductArgs a = {};
  a.p[0] = plan_dense(M, D, N);
  a.p[0].out = static_cast<__nv_bfloat16*>(out);
  a.p[0].partial = static_cast<float*>(partial);
  a.act = act;
  a.bias = static_cast<const __nv_bfloat16*>(bias);
  a.extra = static_cast<const __nv_bfloat16*>(extra);
  a.sums = sums;
  a.dev_err = dev_err;
  Maps tm = {};
  if (!bf16_tile_map(&tm.A[0], x, M, D, kHalf) || !bf16_tile_map(&tm.B[0], w, N, D, kHalf) ||
      !bf16_tile_map(&tm.out, out, M, N, 32) || (extra && !bf16_tile_map(&tm.in, extra, M, N, 32)))
    return SDM_ECUDA;
  if (act == SDM_ACT_SILU) return launch_dense_act<MODE, SDM_ACT_SILU>(tm, a, s);
  if (act == SDM_ACT_GELU) return launch_dense_act<MODE, SDM_ACT_GELU>(tm, a, s);
  if constexpr (MODE == kDense) return launch_dense_act<MODE, SDM_ACT_NONE>(tm, a, s);
  return SDM_EINVAL;
}

// ---- dbias ----

// Sums of dz over the tokens.  The slope pass leaves them for each 32 rows beside dz (dense_sums); without an activation
// dz is dy, and they are taken from there: eight columns a thread and eight lanes of tokens a block.
constexpr int kSumRows = 8;
constexpr int kSumSlice = 256;  // tokens of a block
__global__ void __launch_bounds__(32 * kSumRows) column_sums_kernel(const __nv_bfloat16* dz, int M, int N, int tiles,
                                                                    float* part) {
  __shared__ float sums[kSumRows][32][9];
  wait_previous();
  allow_next();
  const int tile = int(blockIdx.x % unsigned(tiles)), slice = int(blockIdx.x / unsigned(tiles));
  const int col = tile * 256 + int(threadIdx.x) * 8;
  const int m0 = slice * kSumSlice, m_end = min(M - m0, kSumSlice);
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
  if (col < N) {
    const __nv_bfloat16* p = dz + size_t(m0) * N + col;
#pragma unroll 8
    for (int m = int(threadIdx.y); m < m_end; m += kSumRows) {
      float v[8];
      Piece<__nv_bfloat16>::load(*reinterpret_cast<const uint4*>(p + size_t(m) * N), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[threadIdx.y][threadIdx.x][i] = s[i];
  __syncthreads();
  const int id = int(threadIdx.y) * 32 + int(threadIdx.x), c = tile * 256 + id;
  if (c >= N) return;
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) t += sums[i][id / 8][id % 8];
  part[size_t(slice) * N + c] = t;
}
// The rows' sums: 32 columns and 32 lanes of rows a block, each lane's in their order and then the lanes' in theirs.
__global__ void __launch_bounds__(1024) join_sums_kernel(const float* part, int rows, int N, __nv_bfloat16* out) {
  __shared__ float lanes[32][33];
  wait_previous();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < N) {
#pragma unroll 8
    for (int i = int(threadIdx.y); i < rows; i += 32) t += part[size_t(i) * N + c];
  }
  lanes[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y || c >= N) return;
  t = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) t += lanes[i][threadIdx.x];
  out[c] = __float2bfloat16_rn(t);
}
// Rows of partial sums: where the slope pass leaves them, where it does not.
int slope_sum_rows(long long M) { return int((M + 31) / 32); }
int dy_sum_rows(long long M) { return int((M + kSumSlice - 1) / kSumSlice); }

// `rows`: of sums that are there already, or 0.
int launch_column_sums(const void* dz, long long M, int N, float* part, int rows, void* out, cudaStream_t s) {
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!rows) {
    rows = dy_sum_rows(M);
    const int tiles = ceil_div(N, 256);  // slices * tiles: a block has 64 K of dz's elements, which fit on the card
    cfg.gridDim = dim3(unsigned(rows) * unsigned(tiles));
    cfg.blockDim = dim3(32, kSumRows);
    if (cudaLaunchKernelEx(&cfg, column_sums_kernel, static_cast<const __nv_bfloat16*>(dz), int(M), N, tiles, part) !=
        cudaSuccess)
      return SDM_ECUDA;
  }
  cfg.gridDim = dim3(unsigned(ceil_div(N, 32)));
  cfg.blockDim = dim3(32, 32);
  if (cudaLaunchKernelEx(&cfg, join_sums_kernel, static_cast<const float*>(part), rows, N,
                         static_cast<__nv_bfloat16*>(out)) != cudaSuccess)
    return SDM_ECUDA;
  return last_launch_status();
}

int check_dense(const void* x, const void* w, const void* bias, long long M, int D, int N, int act) {
  if (M < 0 || D < 1 || N < 1 || act < SDM_ACT_NONE || act > SDM_ACT_GELU) return SDM_EINVAL;
  if (D % 8 || N % 8 || M > 0x7FFFFFFFLL - 256 || D > 0x3FFFFFFF || N > 0x3FFFFFFF) return SDM_EUNSUPPORTED;
  if (!aligned16(w) || (bias && !aligned16(bias)) || (M > 0 && !aligned16(x))) return SDM_EALIGN;
  return SDM_OK;
}
// Bytes that the gradient's workspace holds: dz where there is an activation, its partial sums, those of dx and dw,
// those of dbias.
struct GradSpace {
  size_t dz, slope, grads, bias;
  GradSpace(long long M, int D, int N, int act) {
    dz = act == SDM_ACT_NONE ? 0 : round256(size_t(M) * N * 2);
    slope = act == SDM_ACT_NONE ? 0 : partial_bytes(plan_dense(int(M), D, N));
    Product p[2];
    plan_grads(int(M), D, N, p);
    grads = partial_bytes(p[0]) + partial_bytes(p[1]);
    bias = round256(size_t(act == SDM_ACT_NONE ? dy_sum_rows(M) : slope_sum_rows(M)) * N * 4);
  }
  size_t total() const { return dz + slope + grads + bias; }
};

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_project_workspace_size(long long M, int D, int N) {
  if (M <= kFewTokens || D < 1 || N < 1 || M > 0x7FFFFFFFLL - 256) return 0;
  return partial_bytes(plan_dense(int(M), D, N));
}

extern "C" int sdm_project(const void* x, const void* w, const void* bias, const void* residual, long long M, int D, int N,
                           int act, void* y, void* workspace, size_t workspace_bytes, int* dev_err, void* stream) {
  const int st = check_dense(x, w, bias, M, D, N, act);
  if (st != SDM_OK) return st;
  if (M == 0) return SDM_OK;
  if (!aligned16(y) || (residual && !aligned16(residual))) return SDM_EALIGN;
  const size_t need = sdm_project_workspace_size(M, D, N);
  if (need && !aligned16(workspace)) return SDM_EALIGN;
  if (workspace_bytes < need) return SDM_ENOSPACE;
  const long long xn = M * D * 2, wn = 2LL * N * D, yn = M * N * 2, sn = (long long)need;
  for (const Extent& e : {dense(x, xn), dense(w, wn), dense(bias, 2LL * N), dense(residual == y ? nullptr : residual, yn)})
    if (meets(e, y, yn) || (need && meets(e, workspace, sn))) return SDM_EOVERLAP;
  if (need && meets(dense(y, yn), workspace, sn)) return SDM_EOVERLAP;
  cudaStream_t s = as_stream(stream);
  if (M <= kFewTokens) {
    if (act == SDM_ACT_SILU) return launch_few_act<SDM_ACT_SILU>(x, w, bias, residual, int(M), D, N, y, s);
    if (act == SDM_ACT_GELU) return launch_few_act<SDM_ACT_GELU>(x, w, bias, residual, int(M), D, N, y, s);
    return launch_few_act<SDM_ACT_NONE>(x, w, bias, residual, int(M), D, N, y, s);
  }
  return launch_dense<kDense>(x, w, bias, residual, int(M), D, N, act, y, workspace, nullptr, dev_err, s);
}

extern "C" size_t sdm_project_backward_workspace_size(long long M, int D, int N, int act) {
  if (M < 1 || D < 1 || N < 1 || M > 0x7FFFFFFFLL - 256) return 0;
  return GradSpace(M, D, N, act).total();
}

extern "C" int sdm_project_backward(const void* x, const void* w, const void* bias, const void* dy, long long M, int D,
                                    int N, int act, void* dx, void* dw, void* dbias, void* workspace,
                                    size_t workspace_bytes, int* dev_err, void* stream) {
  int st = check_dense(x, w, bias, M, D, N, act);
  if (st != SDM_OK) return st;
  if (!aligned16(dw) || (dbias && !aligned16(dbias)) || (M > 0 && (!aligned16(dy) || !aligned16(dx)))) return SDM_EALIGN;
  cudaStream_t s = as_stream(stream);
  const long long xn = M * D * 2, wn = 2LL * N * D, yn = M * N * 2, bn = 2LL * N;
  if (meets(dense(dw, wn), dbias, bn)) return SDM_EOVERLAP;
  for (const Extent& e : {dense(w, wn), dense(bias, bn)})
    if (meets(e, dw, wn) || meets(e, dbias, bn) || meets(e, dx, xn)) return SDM_EOVERLAP;
  if (M == 0) {
    if (cudaMemsetAsync(dw, 0, size_t(wn), s) != cudaSuccess) return SDM_ECUDA;
    return !dbias || cudaMemsetAsync(dbias, 0, size_t(bn), s) == cudaSuccess ? SDM_OK : SDM_ECUDA;
  }
  if (!aligned16(workspace)) return SDM_EALIGN;
  const GradSpace space(M, D, N, act);
  if (workspace_bytes < space.total()) return SDM_ENOSPACE;
  const long long sn = (long long)space.total();
  for (const Extent& e : {dense(x, xn), dense(dy, yn), dense(dx, xn)})
    if (meets(e, dw, wn) || meets(e, dbias, bn) || meets(e, workspace, sn)) return SDM_EOVERLAP;
  for (const Extent& e : {dense(w, wn), dense(bias, bn), dense(dw, wn), dense(dbias, bn)})
    if (meets(e, workspace, sn)) return SDM_EOVERLAP;
  if (meets(dense(x, xn), dx, xn) || meets(dense(dy, yn), dx, xn)) return SDM_EOVERLAP;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  const __nv_bfloat16* dz = static_cast<const __nv_bfloat16*>(dy);
  uint8_t* grads = at + space.dz + space.slope;
  float* sums = reinterpret_cast<float*>(grads + space.grads);
  int rows = 0;
  if (act != SDM_ACT_NONE) {
    st = launch_dense<kDenseSlope>(x, w, bias, dy, int(M), D, N, act, at, at + space.dz, dbias ? sums : nullptr, dev_err, s);
    if (st != SDM_OK) return st;
    dz = reinterpret_cast<const __nv_bfloat16*>(at);
    if (!space.slope) rows = slope_sum_rows(M);  // a product that is joined leaves none
  }
  st = launch_grads(dz, x, w, int(M), D, N, dx, dw, grads, dev_err, s);
  if (st != SDM_OK || !dbias) return st;
  return launch_column_sums(dz, M, N, sums, rows, dbias, s);
}
