// The norms after and before a block in one pass, with the block's gate, residual scale and residual:
//
//   a = x / rms(x) * after * act(gate)     rms over each of `groups` groups of channels
//   r = residual + scale * a
//   y = r / rms(r) * weight                rms(v) = sqrt(mean(v^2) + eps)
//
// any part of which may be absent.  HBM bounds it: a row is read once into registers, and both sums over it are taken there in
// fp32 (a norm by itself, a gate and a residual addition would each read and write it again).  A row has 8 to 1024 threads
// of eight channels; a block of 128 threads has several short rows.  Blocks stay and take rows in turn, the next one on its way
// while one is worked on.  16,384 rows of 2048 with both norms, scale and an fp32 stream: 66 us, 0.90
// of the HBM floor; 16,384 x 16 groups of 128 with a gate 37.5 (0.79).  4 rows: 5.9, a launch.
#include "sdm_norm.cuh"

namespace sdm {
namespace {

struct Forward {
  sdm_norm_args io;
  void *y, *r;
  int slots;  // teams of a group
};

constexpr int kThreads = 1024;  // of an SM

template <typename TX, typename TR, int TPR, int P, bool VEC>
__global__ void __launch_bounds__(norm_block(TPR), kThreads / norm_block(TPR)) norm_kernel(const __grid_constant__ Forward a) {
  typedef Row<TPR, P, VEC> R;
  constexpr int E = R::E, RPB = norm_block(TPR) / TPR, W = norm_block(TPR) / 32;
  // Rows on 16 bytes are faster with one way through the loop (16,384 x 2048: 66 us and 68).
  constexpr bool kBreak = R::kAlone && !VEC;
  __shared__ float part[2][2][W][1];
  __shared__ Kept<R, norm_block(TPR), 3> kept;
  const sdm_norm_args& io = a.io;
  const int t = threadIdx.x % TPR, n = io.D / io.groups;
  const float rn = 1.0f / float(n);
  const unsigned team = blockIdx.x * RPB + threadIdx.x / TPR;
  const unsigned slot = team / unsigned(io.groups), group = team % unsigned(io.groups);
  const bool used = slot < unsigned(a.slots);
  const long long off = (long long)group * n, at = used ? off : 0;
  const int mine = used ? n : 0;

  // A row as it lies in memory; the next one is asked for while this one is worked on.
  typename R::template Raw<TX> rx, rz;
  typename R::template Raw<TR> rs;
  const TX* px = static_cast<const TX*>(io.x) + slot * io.x_rs + off;
  const TX* pz = static_cast<const TX*>(io.gate) + (io.gate ? slot * io.gate_rs + off : 0);
  const TR* ps = static_cast<const TR*>(io.residual) + (io.residual ? slot * io.residual_rs + off : 0);
  const long long out = slot * (long long)io.D + off, step = a.slots * (long long)io.D;
  TX* y = static_cast<TX*>(a.y) + (a.y ? out : 0);
  TR* r = static_cast<TR*>(a.r) + (a.r ? out : 0);
  auto ask = [&](long long m0) {
    if (kBreak && m0 + slot >= io.M) return;
    const int cols = kBreak || (used && m0 + slot < io.M) ? n : 0;
    rx.ask(px, t, cols), px += a.slots * io.x_rs;
    if (io.gate) rz.ask(pz, t, cols), pz += a.slots * io.gate_rs;
    if (io.residual) rs.ask(ps, t, cols), ps += a.slots * io.residual_rs;
  };
  ask(0);
  if (io.after) kept.put(0, io.after, io.w_dtype, at, t, mine);
  if (io.scale) kept.put(1, io.scale, io.w_dtype, at, t, mine);
  if (a.y) kept.put(2, io.weight, io.w_dtype, at, t, mine);

  int turn = 0;
  for (long long m0 = 0; m0 < io.M; m0 += a.slots, turn ^= 1) {
    if (kBreak && m0 + slot >= io.M) break;
    const int cols = kBreak || (used && m0 + slot < io.M) ? n : 0;
    float v[E], s[E], z[E], w[E];
    rx.get(v);
    if (io.gate) rz.get(z);
    if (io.residual) rs.get(s);
    if (m0 + a.slots < io.M) ask(m0 + a.slots);
    if (io.after) {
      float q[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) q[0] = fmaf(v[e], v[e], q[0]);
      row_sums<TPR>(q, part[turn][0]);
      const float inv = rsqrtf(fmaf(q[0], rn, io.eps));
      kept.get(0, io.after, io.w_dtype, at, t, mine, w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= inv * w[e];
    }
    if (io.gate) {
      if (io.act == SDM_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= silu(z[e]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] *= z[e];
      }
    }
    if (io.scale) {
      kept.get(1, io.scale, io.w_dtype, at, t, mine, w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= w[e];
    }
    if (io.residual) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += s[e];
    }
    if (a.r) R::store(r, t, cols, v), r += step;
    if (a.y) {
      float q[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) q[0] = fmaf(v[e], v[e], q[0]);
      row_sums<TPR>(q, part[turn][1]);
      const float inv = rsqrtf(fmaf(q[0], rn, io.eps));
      kept.get(2, io.weight, io.w_dtype, at, t, mine, w);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] *= inv * w[e];
      R::store(y, t, cols, v), y += step;
    }
  }
}

template <typename TX, typename TR, bool VEC>
int launch(Forward a, cudaStream_t s) {
  return norm_by_width<1024>(a.io.D / a.io.groups, [&](auto tpr, auto pieces) {
    constexpr int block = norm_block(tpr), RPB = block / int(tpr);
    // Teams of a group: as many as the card holds at once, and no more than there are rows.
    const long long most = 152LL * (kThreads / block) * RPB / a.io.groups, slots = most < 1 ? 1 : most;
    a.slots = int(slots < a.io.M ? slots : a.io.M);
    const long long teams = (long long)a.slots * a.io.groups;
    norm_kernel<TX, TR, tpr, pieces, VEC><<<unsigned((teams + RPB - 1) / RPB), block, 0, s>>>(a);
    return last_launch_status();
  });
}
template <typename TX, typename TR>
int launch(const Forward& a, bool vec, cudaStream_t s) {
  return vec ? launch<TX, TR, true>(a, s) : launch<TX, TR, false>(a, s);
}

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
  const Forward a{io, y, r, 0};
  cudaStream_t s = as_stream(stream);
  if (io.x_dtype == SDM_F32) return launch<float, float>(a, vec, s);
  return io.r_dtype == SDM_F32 ? launch<__nv_bfloat16, float>(a, vec, s) : launch<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
}
