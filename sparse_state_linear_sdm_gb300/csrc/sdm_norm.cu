// The norms after and before a block in one pass, with the block's gate, residual scale and residual:
//
//   a = x / rms(x) * after * act(gate)     rms over each of `groups` groups of channels
//   r = residual + scale * a
//   y = r / rms(r) * weight                rms(v) = sqrt(mean(v^2) + eps)
//
// any part of which may be absent.  HBM bounds it: a row is read once into registers, and both sums over it are taken there in
// fp32 (a norm by itself, a gate and a residual addition would each read and write it again).  A row has 8 to 512 threads, at
// most 32 channels each; a block of 128 threads has several short rows.  The weights come from L1.
#include "sdm_norm.cuh"

namespace sdm {
namespace {

struct Forward {
  sdm_norm_args io;
  void *y, *r;
};

template <typename TX, typename TR, int TPR, int P, bool VEC>
__global__ void __launch_bounds__(norm_block(TPR)) norm_kernel(const __grid_constant__ Forward a) {
  typedef Row<TPR, P, VEC> R;
  constexpr int E = R::E, RPB = norm_block(TPR) / TPR, W = norm_block(TPR) / 32;
  __shared__ float part[2][W][1];
  const sdm_norm_args& io = a.io;
  const int t = threadIdx.x % TPR, n = io.D / io.groups;
  const unsigned row = blockIdx.x * RPB + threadIdx.x / TPR, rows = unsigned(io.M) * unsigned(io.groups);
  const bool live = row < rows;
  const long long m = live ? row / unsigned(io.groups) : 0;
  const long long off = live ? (long long)(row % unsigned(io.groups)) * n : 0;
  const int cols = live ? n : 0;

  float v[E], s[E], z[E], w[E];
  R::load(static_cast<const TX*>(io.x) + m * io.x_rs + off, t, cols, v);
  if (io.residual) R::load(static_cast<const TR*>(io.residual) + m * io.residual_rs + off, t, cols, s);
  if (io.gate) R::load(static_cast<const TX*>(io.gate) + m * io.gate_rs + off, t, cols, z);
  if (io.after) {
    R::weights(io.after, io.w_dtype, off, t, cols, w);
    float q[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) q[0] = fmaf(v[e], v[e], q[0]);
    row_sums<TPR>(q, part[0]);
    const float inv = rsqrtf(q[0] / float(n) + io.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= inv * w[e];
  }
  if (io.gate) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= io.act == SDM_ACT_SILU ? silu(z[e]) : z[e];
  }
  if (io.scale) {
    R::weights(io.scale, io.w_dtype, off, t, cols, w);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= w[e];
  }
  if (io.residual) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] += s[e];
  }
  if (a.r) R::store(static_cast<TR*>(a.r) + m * io.D + off, t, cols, v);
  if (a.y) {
    R::weights(io.weight, io.w_dtype, 0, t, cols, w);
    float q[1] = {0.f};
#pragma unroll
    for (int e = 0; e < E; ++e) q[0] = fmaf(v[e], v[e], q[0]);
    row_sums<TPR>(q, part[1]);
    const float inv = rsqrtf(q[0] / float(n) + io.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] *= inv * w[e];
    R::store(static_cast<TX*>(a.y) + m * io.D, t, cols, v);
  }
}

template <typename TX, typename TR, int TPR, int P, bool VEC>
struct Launch {
  static int run(const Forward& a, cudaStream_t s) {
    constexpr int block = norm_block(TPR), RPB = block / TPR;
    const long long rows = a.io.M * a.io.groups;
    norm_kernel<TX, TR, TPR, P, VEC><<<unsigned((rows + RPB - 1) / RPB), block, 0, s>>>(a);
    return last_launch_status();
  }
};

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int sdm_residual_norm(const sdm_norm_args* args, void* y, void* r, void* stream) {
  if (!args) return SDM_EINVAL;
  const sdm_norm_args& io = *args;
  const int st = check_norm(io);
  if (st != SDM_OK) return st;
  if ((y != nullptr) != (io.weight != nullptr) || (!y && !r)) {
    if (io.M > 0) return SDM_EINVAL;
  }
  if (io.M == 0) return SDM_OK;
  const uintptr_t ox = norm_odd(io.x_dtype), orr = norm_odd(io.r_dtype);
  if (!io.x || misaligned(io.x, ox) || misaligned(io.gate, ox) || misaligned(y, ox) || misaligned(io.residual, orr) ||
      misaligned(r, orr))
    return SDM_EALIGN;
  const int ex = norm_es(io.x_dtype), er = norm_es(io.r_dtype), ew = norm_es(io.w_dtype);
  const Extent in[] = {norm_rows(io.x, io.M, io.x_rs, io.D, ex), norm_rows(io.gate, io.M, io.gate_rs, io.D, ex),
                       norm_rows(io.residual, io.M, io.residual_rs, io.D, er)};
  const long long yr = (long long)io.D * ex, rr = (long long)io.D * er;
  for (const Extent& e : in)
    if ((!same_rows(e, y, yr) && meets(e, y, io.M * yr)) || (!same_rows(e, r, rr) && meets(e, r, io.M * rr)))
      return SDM_EOVERLAP;
  for (const void* w : {io.after, io.scale, io.weight})
    if (meets(dense(w, (long long)io.D * ew), y, io.M * yr) || meets(dense(w, (long long)io.D * ew), r, io.M * rr))
      return SDM_EOVERLAP;
  if (meets(dense(y, io.M * yr), r, io.M * rr)) return SDM_EOVERLAP;
  auto rows16 = [](const void* p, long long rs) { return !misaligned(p, 15) && rs % 8 == 0; };
  const bool vec = (io.D / io.groups) % 8 == 0 && rows16(io.x, io.x_rs) && rows16(io.gate, io.gate_rs) &&
                   rows16(io.residual, io.residual_rs) && !misaligned(y, 15) && !misaligned(r, 15) &&
                   !misaligned(io.after, 15) && !misaligned(io.scale, 15) && !misaligned(io.weight, 15);
  return norm_dispatch<Launch>(io.x_dtype, io.r_dtype, vec, io.D / io.groups, Forward{io, y, r}, as_stream(stream));
}
