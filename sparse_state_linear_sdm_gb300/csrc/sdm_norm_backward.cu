// Gradient of the norms (sdm_norm.cu).  With i = 1 / rms(r), j = 1 / rms(x), n = x j after, s = act(gate):
//
//   d  = dr + i (dy weight - r i^2 mean(dy weight r))          the stream's gradient, and the residual's
//   dweight = sum dy r i,   dscale = sum d n s
//   u  = d scale,   dgate = u n act'(gate),   dafter = sum u s x j
//   dx = j (u s after - x j^2 mean(u s after x))
//
// The forward pass keeps r; everything else is formed again from x and the gate, which costs no byte that the gradient would not
// read anyway.  HBM bounds it.  A row is in registers as in the forward pass.  Blocks stay and take rows in turn, so that the sums
// over rows run in registers as well; each team of threads keeps to one group of channels, writes its sums once, and
// a second kernel adds the teams' in a fixed order: results do not depend on timing.
#include "sdm_norm.cuh"

namespace sdm {
namespace {

struct Backward {
  sdm_norm_args io;
  const void *r, *dy, *dr;
  long long r_rs, dy_rs, dr_rs;
  void *dx, *dres, *dgate;
  void *dafter, *dscale, *dweight;
  float* part;  // [slots][kinds][D]
  int slots;    // teams of a group
  int kinds;    // sums wanted
};

template <typename TX, typename TR, int TPR, int P, bool VEC>
__global__ void __launch_bounds__(norm_block(TPR)) backward_kernel(const __grid_constant__ Backward a) {
  typedef Row<TPR, P, VEC> R;
  constexpr int E = R::E, RPB = norm_block(TPR) / TPR, W = norm_block(TPR) / 32;
  __shared__ float part1[2][W][3], part2[2][W][1];
  const sdm_norm_args& io = a.io;
  const int t = threadIdx.x % TPR, n = io.D / io.groups;
  const unsigned team = blockIdx.x * RPB + threadIdx.x / TPR;
  const unsigned slot = team / unsigned(io.groups), group = team % unsigned(io.groups);
  const bool used = slot < unsigned(a.slots);
  const long long off = (long long)group * n;
  allow_next();

  float sum_after[E], sum_scale[E], sum_weight[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum_after[e] = sum_scale[e] = sum_weight[e] = 0.f;

  int turn = 0;
  for (long long m0 = 0; m0 < io.M; m0 += a.slots, turn ^= 1) {
    const bool live = used && m0 + slot < io.M;
    const long long m = live ? m0 + slot : 0;
    const long long at = live ? off : 0;
    const int cols = live ? n : 0;
    float x[E], z[E], r[E], d[E], dr[E], w[E];
    const bool inner = a.dx != nullptr || a.dgate || a.dafter || a.dscale;
    if (io.after || io.gate || io.scale) R::load(static_cast<const TX*>(io.x) + m * io.x_rs + at, t, cols, x);
    if (io.gate) R::load(static_cast<const TX*>(io.gate) + m * io.gate_rs + at, t, cols, z);
    if (a.dy) {
      R::load(static_cast<const TX*>(a.dy) + m * a.dy_rs + at, t, cols, d);
      R::load(static_cast<const TR*>(a.r) + m * a.r_rs + at, t, cols, r);
    }
    if (a.dr) R::load(static_cast<const TR*>(a.dr) + m * a.dr_rs + at, t, cols, dr);

    float q[3] = {0.f, 0.f, 0.f};
    if (a.dy) {
      R::weights(io.weight, io.w_dtype, at, t, cols, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[0] = fmaf(r[e], r[e], q[0]);
        q[1] = fmaf(d[e] * w[e], r[e], q[1]);
      }
    }
    if (io.after) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[2] = fmaf(x[e], x[e], q[2]);
    }
    if (a.dy || io.after) row_sums<TPR>(q, part1[turn]);
    if (a.dy) {
      const float i = live ? rsqrtf(q[0] / float(n) + io.eps) : 0.f, c = i * i * (q[1] / float(n));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sum_weight[e] = fmaf(d[e], r[e] * i, sum_weight[e]);
        d[e] = i * (d[e] * w[e] - r[e] * c);
        if (a.dr) d[e] += dr[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = dr[e];
    }
    if (a.dres) R::store(static_cast<TR*>(a.dres) + m * io.D + at, t, cols, d);
    if (!inner) continue;

    float j = 1.f;
    if (io.after) {
      j = live ? rsqrtf(q[2] / float(n) + io.eps) : 0.f;
      R::weights(io.after, io.w_dtype, at, t, cols, w);
    }
    if (io.scale) {
      float c[E];
      R::weights(io.scale, io.w_dtype, at, t, cols, c);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float o = io.after ? x[e] * j * w[e] : x[e];
        if (io.gate) o *= io.act == SDM_ACT_SILU ? silu(z[e]) : z[e];
        sum_scale[e] = fmaf(d[e], o, sum_scale[e]);
        d[e] *= c[e];
      }
    }
    if (io.gate) {
      float dz[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float o = io.after ? x[e] * j * w[e] : x[e];
        float s = z[e], ds = 1.f;
        if (io.act == SDM_ACT_SILU) {
          const float p = sigmoid(z[e]);
          s = z[e] * p;
          ds = fmaf(s, 1.f - p, p);
        }
        dz[e] = d[e] * o * ds;
        d[e] *= s;
      }
      if (a.dgate) R::store(static_cast<TX*>(a.dgate) + m * io.D + at, t, cols, dz);
    }
    if (io.after) {
      float g[1] = {0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sum_after[e] = fmaf(d[e], x[e] * j, sum_after[e]);
        d[e] *= w[e];
        g[0] = fmaf(d[e], x[e], g[0]);
      }
      row_sums<TPR>(g, part2[turn]);
      const float c = j * j * (g[0] / float(n));
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = j * (d[e] - x[e] * c);
    }
    if (a.dx) R::store(static_cast<TX*>(a.dx) + m * io.D + at, t, cols, d);
  }
  if (!used) return;
  float* p = a.part + (long long)slot * a.kinds * io.D + off;
  if (a.dafter) R::store(p, t, n, sum_after), p += io.D;
  if (a.dscale) R::store(p, t, n, sum_scale), p += io.D;
  if (a.dweight) R::store(p, t, n, sum_weight);
}

// Adds the teams' sums: a block has 32 columns and 32 lanes of teams, each lane's in their order and then the
// lanes' in theirs.
__global__ void __launch_bounds__(1024) sums_kernel(const __grid_constant__ Backward a) {
  __shared__ float part[32][33];
  wait_previous();
  const int D = a.io.D, c = blockIdx.x * 32 + threadIdx.x, lane = threadIdx.y, kind = blockIdx.y;
  float s = 0.f;
  if (c < D) {
#pragma unroll 4
    for (int i = lane; i < a.slots; i += 32) s += a.part[((long long)i * a.kinds + kind) * D + c];
  }
  part[lane][threadIdx.x] = s;
  __syncthreads();
  if (lane || c >= D) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
  int k = kind;
  void* out = nullptr;
  for (void* o : {a.dafter, a.dscale, a.dweight})
    if (o && k-- == 0) out = o;
  if (a.io.w_dtype == SDM_F32)
    static_cast<float*>(out)[c] = s;
  else
    static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
}

// Teams of a group: as many as keep the card busy and no more than there are rows.  The blocks of an SM are as many
// as 128 registers a thread allow.
int slots_for(long long M, int D, int groups) {
  const int n = D / groups, tpr = n <= 64 ? 8 : n <= 128 ? 16 : n <= 256 ? 32 : n <= 1024 ? 64 : n <= 2048 ? 128 : n <= 4096 ? 256 : 512;
  const int block = norm_block(tpr), teams = 152 * (512 / block) * (block / tpr);
  long long s = teams / groups;
  if (s < 1) s = 1;
  return int(s < M ? s : M);
}

template <typename TX, typename TR, int TPR, int P, bool VEC>
struct Launch {
  static int run(const Backward& a, cudaStream_t s) {
    constexpr int block = norm_block(TPR), RPB = block / TPR;
    const long long teams = (long long)a.slots * a.io.groups;
    backward_kernel<TX, TR, TPR, P, VEC><<<unsigned((teams + RPB - 1) / RPB), block, 0, s>>>(a);
    return last_launch_status();
  }
};

int launch_sums(const Backward& a, cudaStream_t s) {
  if (!a.kinds) return SDM_OK;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.io.D + 31) / 32), unsigned(a.kinds));
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.io.M > 0 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, sums_kernel, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_residual_norm_backward_workspace_size(long long M, int D, int groups) {
  if (M < 1 || D < 1 || groups < 1 || D % groups || D / groups > kNormMax) return 0;
  return size_t(slots_for(M, D, groups)) * 3 * D * 4;
}

extern "C" int sdm_residual_norm_backward(const sdm_norm_args* args, const sdm_norm_grads* grads, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (!args || !grads) return SDM_EINVAL;
  const sdm_norm_args& io = *args;
  const sdm_norm_grads& g = *grads;
  const int st = check_norm(io);
  if (st != SDM_OK) return st;
  if ((g.dafter && !io.after) || (g.dscale && !io.scale) || (g.dweight && !io.weight) || (g.dgate && !io.gate))
    return SDM_EINVAL;
  Backward a = {};
  a.io = io;
  a.kinds = (g.dafter != nullptr) + (g.dscale != nullptr) + (g.dweight != nullptr);
  a.dafter = g.dafter, a.dscale = g.dscale, a.dweight = g.dweight;
  const uintptr_t ow = norm_odd(io.w_dtype);
  if (misaligned(g.dafter, ow) || misaligned(g.dscale, ow) || misaligned(g.dweight, ow)) return SDM_EALIGN;
  const int ex = norm_es(io.x_dtype), er = norm_es(io.r_dtype), ew = norm_es(io.w_dtype);
  const long long wn = (long long)io.D * ew;
  cudaStream_t s = as_stream(stream);
  if (io.M == 0) return launch_sums(a, s);
  if ((io.weight != nullptr) != (g.dy != nullptr) || (!g.dy && !g.dr) || (g.dy && !g.r)) return SDM_EINVAL;
  if (!io.x && (io.after || io.gate || io.scale)) return SDM_EINVAL;
  const uintptr_t ox = norm_odd(io.x_dtype), orr = norm_odd(io.r_dtype);
  for (const void* p : {io.x, io.gate, g.dy, (const void*)g.dx, (const void*)g.dgate})
    if (misaligned(p, ox)) return SDM_EALIGN;
  for (const void* p : {g.r, g.dr, (const void*)g.dresidual})
    if (misaligned(p, orr)) return SDM_EALIGN;
  const size_t need = a.kinds ? sdm_residual_norm_backward_workspace_size(io.M, io.D, io.groups) : 0;
  if (need) {
    if (!aligned16(workspace)) return SDM_EALIGN;
    if (workspace_bytes < need) return SDM_ENOSPACE;
  }
  const long long xr = (long long)io.D * ex, rr = (long long)io.D * er, wsn = (long long)need;
  struct Out {
    const void* p;
    long long row;
  };
  const Out out[] = {{g.dx, xr}, {g.dgate, xr}, {g.dresidual, rr}};
  const void* sums[] = {g.dafter, g.dscale, g.dweight};
  const Extent in[] = {norm_rows(io.x, io.M, io.x_rs, io.D, ex), norm_rows(io.gate, io.M, io.gate_rs, io.D, ex),
                       norm_rows(g.dy, io.M, g.dy_rs, io.D, ex), norm_rows(g.r, io.M, g.r_rs, io.D, er),
                       norm_rows(g.dr, io.M, g.dr_rs, io.D, er)};
  const Extent weights[] = {dense(io.after, wn), dense(io.scale, wn), dense(io.weight, wn)};
  for (int i = 0; i < 3; ++i) {
    for (const Extent& e : in) {
      if (!same_rows(e, out[i].p, out[i].row) && meets(e, out[i].p, io.M * out[i].row)) return SDM_EOVERLAP;
      if (meets(e, sums[i], wn)) return SDM_EOVERLAP;
    }
    for (const Extent& e : weights)
      if (meets(e, out[i].p, io.M * out[i].row) || meets(e, sums[i], wn)) return SDM_EOVERLAP;
    for (int k = 0; k < 3; ++k) {
      if (k != i && meets(dense(out[k].p, io.M * out[k].row), out[i].p, io.M * out[i].row)) return SDM_EOVERLAP;
      if (k != i && meets(dense(sums[k], wn), sums[i], wn)) return SDM_EOVERLAP;
      if (meets(dense(sums[k], wn), out[i].p, io.M * out[i].row)) return SDM_EOVERLAP;
    }
    if (need && (meets(dense(out[i].p, io.M * out[i].row), workspace, wsn) || meets(dense(sums[i], wn), workspace, wsn) ||
                 meets(weights[i], workspace, wsn)))
      return SDM_EOVERLAP;
  }
  for (const Extent& e : in)
    if (need && meets(e, workspace, wsn)) return SDM_EOVERLAP;

  a.r = g.r, a.dy = g.dy, a.dr = g.dr;
  a.r_rs = g.r_rs, a.dy_rs = g.dy_rs, a.dr_rs = g.dr_rs;
  a.dx = g.dx, a.dres = g.dresidual, a.dgate = g.dgate;
  a.part = static_cast<float*>(workspace);
  a.slots = slots_for(io.M, io.D, io.groups);
  auto rows16 = [](const void* p, long long rs) { return !misaligned(p, 15) && rs % 8 == 0; };
  const bool vec = (io.D / io.groups) % 8 == 0 && rows16(io.x, io.x_rs) && rows16(io.gate, io.gate_rs) &&
                   rows16(g.dy, g.dy_rs) && rows16(g.r, g.r_rs) && rows16(g.dr, g.dr_rs) && !misaligned(g.dx, 15) &&
                   !misaligned(g.dgate, 15) && !misaligned(g.dresidual, 15) && !misaligned(io.after, 15) &&
                   !misaligned(io.scale, 15) && !misaligned(io.weight, 15);
  const int r = norm_dispatch<Launch>(io.x_dtype, io.r_dtype, vec, io.D / io.groups, a, s);
  return r != SDM_OK ? r : launch_sums(a, s);
}
