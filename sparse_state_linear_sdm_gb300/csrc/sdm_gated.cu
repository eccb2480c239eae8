// Gated feed-forward projections and their gradient, on the tcgen05 tensor cores (sdm_product.cuh).
//
//   g = x Wg^T,  u = x Wu^T,  h = act(g) * u                     (w = [Wg; Wu], [2F, D])
//   dg = dh * u * act'(g),  du = dh * act(g)
//   dx = dg Wg + du Wu = [dg | du] w,   dw = [dg | du]^T x
//
// Sums are fp32; dg and du are the only rounding between inputs and outputs: the tensor cores take them
// at full rate as bf16, like x and w beside them, and at half of it or less, with twice the bytes to hold
// and read, in anything wider.  Each is half a unit of bf16 off, so dx and dw are 0.0023 of their norm off
// where their own rounding alone makes 0.0017.
//
// The tensor pipe bounds the large cases, and the card's power: 16,384 tokens of 2048 x 8192 take
// 0.62 to 0.64 ms back to back (1,720 to 1,780 TFLOP/s), the gradient of 32,768 tokens 4.17 to 4.27 ms
// (1,545 to 1,580; 1,750 in ten calls from idle).  Neither the forward nor the slope pass splits its
// reduction, so few tiles leave pairs idle: 256 tokens of 2048 x 1024 are 8 units and take 16.8 us.
#include "sdm_product.cuh"

namespace sdm {
namespace {

// ---- few tokens ----
//
// A decode step's product reads all of w for a handful of tokens: HBM bounds it, and what counts is
// that every SM reads its even share with enough loads under way.  A block takes 8 columns f: the 8
// rows of Wg and the 8 of Wu are the 16 rows of one mma.m16n8k16, tokens its 8 columns, so that a lane
// ends with g and u of the same elements.  Each of the four warps takes runs of 8 K steps of 32 (512
// bytes of a row: 14.5 us at 4 tokens of 2048 x 8192 where the warps take single steps in turn, 12.8
// so), straight from global memory in 16-byte words (a lane's 8 consecutive k stand for the two groups
// of four that it holds of two MMAs; x is read the same way, so the order of k is the same on both
// sides), and their sums meet in shared memory.
constexpr int kFewThreads = 128;
constexpr int kFewF = 8;
// NT groups of 8 tokens.
template <int ACT, int NT>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const __nv_bfloat16* __restrict__ x,
                                                          const __nv_bfloat16* __restrict__ w, int M,
                                                          int D, int F, __nv_bfloat16* h) {
  constexpr int kWarps = kFewThreads / 32, kAhead = 8 / NT;
  __shared__ float4 part[kWarps][NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int f = blockIdx.x * kFewF + g;  // F % 8 == 0
  const __nv_bfloat16* wg = w + size_t(f) * D + c * 8;
  const __nv_bfloat16* wu = wg + size_t(F) * D;
  const __nv_bfloat16* xr = x + size_t(g) * D + c * 8;

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = warp * 32 * kAhead; k0 < D; k0 += kWarps * 32 * kAhead) {
    uint4 vg[kAhead], vu[kAhead], vx[kAhead][NT];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j * 32;
      const bool in = k + c * 8 < D;  // D % 8 == 0
      vg[j] = in ? load_stream(wg + k) : zero;
      vu[j] = in ? load_stream(wu + k) : zero;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        vx[j][t] = in && t * 8 + g < M ? *reinterpret_cast<const uint4*>(xr + size_t(t) * 8 * D + k) : zero;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma16n8(acc[t], vg[j].x, vu[j].x, vg[j].y, vu[j].y, vx[j][t].x, vx[j][t].y);
        mma16n8(acc[t], vg[j].z, vu[j].z, vg[j].w, vu[j].w, vx[j][t].z, vx[j][t].w);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) part[warp][t][lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
  __syncthreads();
  for (int t = warp; t < NT; t += kWarps) {  // g of tokens 2c, 2c+1 in x, y; u in z, w
    float4 s = part[0][t][lane];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) {
      const float4 p = part[i][t][lane];
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    const int m = t * 8 + 2 * c;
    if (m < M) h[size_t(m) * F + f] = __float2bfloat16_rn(gate<ACT>(s.x) * s.z);
    if (m + 1 < M) h[size_t(m + 1) * F + f] = __float2bfloat16_rn(gate<ACT>(s.y) * s.w);
  }
}

template <int ACT>
int launch_few(const void* x, const void* w, int M, int D, int F, void* h, cudaStream_t s) {
  const __nv_bfloat16* xp = static_cast<const __nv_bfloat16*>(x);
  const __nv_bfloat16* wp = static_cast<const __nv_bfloat16*>(w);
  __nv_bfloat16* hp = static_cast<__nv_bfloat16*>(h);
  const unsigned blocks = unsigned(F / kFewF);
  if (M <= 8)
    few_kernel<ACT, 1><<<blocks, kFewThreads, 0, s>>>(xp, wp, M, D, F, hp);
  else
    few_kernel<ACT, 2><<<blocks, kFewThreads, 0, s>>>(xp, wp, M, D, F, hp);
  return last_launch_status();
}

template <int MODE>
int launch_act(const Maps& tm, const ProductArgs& a, cudaStream_t s) {
  return a.act == SDM_ACT_SILU ? launch_mode<MODE, SDM_ACT_SILU>(tm, a, s)
                               : launch_mode<MODE, SDM_ACT_GELU>(tm, a, s);
}

int check_gated(const void* x, const void* w, long long M, int D, int F, int act) {
  if (M < 0 || D < 1 || F < 1 || (act != SDM_ACT_SILU && act != SDM_ACT_GELU)) return SDM_EINVAL;
  if (D % 8 || F % 8 || M > 0x7FFFFFFFLL - 256 || D > 0x3FFFFFF || F > 0x3FFFFFF) return SDM_EUNSUPPORTED;
  if (!aligned16(w) || (M > 0 && !aligned16(x))) return SDM_EALIGN;
  return SDM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int sdm_project_gated(const void* x, const void* w, long long M, int D, int F, int act,
                                 void* h, int* dev_err, void* stream) {
  const int st = check_gated(x, w, M, D, F, act);
  if (st != SDM_OK) return st;
  if (M == 0) return SDM_OK;
  if (!aligned16(h)) return SDM_EALIGN;
  const long long hn = M * F * 2;
  if (meets(dense(x, M * D * 2), h, hn) || meets(dense(w, 4LL * F * D), h, hn)) return SDM_EOVERLAP;
  if (M <= kFewTokens)
    return act == SDM_ACT_SILU ? launch_few<SDM_ACT_SILU>(x, w, int(M), D, F, h, as_stream(stream))
                               : launch_few<SDM_ACT_GELU>(x, w, int(M), D, F, h, as_stream(stream));
  Maps tm = {};
  if (!bf16_tile_map(&tm.A[0], x, int(M), D, kHalf) || !bf16_tile_map(&tm.B[0], w, F, D, kHalf) ||
      !bf16_tile_map(&tm.B[1], static_cast<const __nv_bfloat16*>(w) + size_t(F) * D, F, D, kHalf) ||
      !bf16_tile_map(&tm.out, h, int(M), F, 32))
    return SDM_ECUDA;
  ProductArgs a = {};
  a.p[0] = product(int(M), F, kHalf, D);
  a.act = act;
  a.dev_err = dev_err;
  return launch_act<kForward>(tm, a, as_stream(stream));
}

extern "C" size_t sdm_project_gated_backward_workspace_size(long long M, int D, int F) {
  if (M < 1 || D < 1 || F < 1 || M > 0x7FFFFFFFLL - 256) return 0;
  Product p[2];
  plan_grads(int(M), D, 2 * F, p);
  return round256(size_t(M) * 2 * F * 2) + partial_bytes(p[0]) + partial_bytes(p[1]);
}

extern "C" int sdm_project_gated_backward(const void* x, const void* w, const void* dh, long long M,
                                          int D, int F, int act, void* dx, void* dw, void* workspace,
                                          size_t workspace_bytes, int* dev_err, void* stream) {
  int st = check_gated(x, w, M, D, F, act);
  if (st != SDM_OK) return st;
  if (!aligned16(dw) || (M > 0 && (!aligned16(dh) || !aligned16(dx)))) return SDM_EALIGN;
  cudaStream_t s = as_stream(stream);
  const long long xn = M * D * 2, wn = 4LL * F * D;
  if (M == 0 && meets(dense(w, wn), dw, wn)) return SDM_EOVERLAP;
  if (M == 0)
    return cudaMemsetAsync(dw, 0, size_t(2) * F * D * 2, s) == cudaSuccess ? SDM_OK : SDM_ECUDA;
  if (!aligned16(workspace)) return SDM_EALIGN;
  const size_t need = sdm_project_gated_backward_workspace_size(M, D, F);
  if (workspace_bytes < need) return SDM_ENOSPACE;
  for (const Extent& e : {dense(x, xn), dense(w, wn), dense(workspace, (long long)need)})
    if (meets(e, dx, xn) || meets(e, dw, wn)) return SDM_EOVERLAP;
  if (meets(dense(dx, xn), dw, wn)) return SDM_EOVERLAP;
  for (const Extent& e : {dense(x, xn), dense(w, wn), dense(dh, M * F * 2)})
    if (meets(e, workspace, (long long)need)) return SDM_EOVERLAP;
  __nv_bfloat16* slope = static_cast<__nv_bfloat16*>(workspace);  // [dg | du], [M, 2F]
  Maps ts = {};
  if (!bf16_tile_map(&ts.A[0], x, int(M), D, kHalf) || !bf16_tile_map(&ts.B[0], w, F, D, kHalf) ||
      !bf16_tile_map(&ts.B[1], static_cast<const __nv_bfloat16*>(w) + size_t(F) * D, F, D, kHalf) ||
      !bf16_tile_map(&ts.in, dh, int(M), F, 32) || !bf16_tile_map(&ts.out, slope, int(M), F, 32, 2LL * F) ||
      !bf16_tile_map(&ts.out2, slope + F, int(M), F, 32, 2LL * F))
    return SDM_ECUDA;
  ProductArgs as = {};
  as.p[0] = product(int(M), F, kHalf, D);
  as.act = act;
  as.dev_err = dev_err;
  st = launch_act<kSlope>(ts, as, s);
  if (st != SDM_OK) return st;
  return launch_grads(slope, x, w, int(M), D, 2 * F, dx, dw,
                      static_cast<uint8_t*>(workspace) + round256(size_t(M) * 2 * F * 2), dev_err, s);
}
