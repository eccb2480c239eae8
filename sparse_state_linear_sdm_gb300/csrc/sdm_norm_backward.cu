// Gradient of the norms: checks, the sums over rows, and the instances of one pair of types (sdm_norm_backward.cuh; the
// others are in sdm_norm_backward_mixed.cu and sdm_norm_backward_f32.cu, so that they compile side by side).
#include "sdm_norm_backward.cuh"
#include "sdm_tcgen05.cuh"

namespace sdm {

extern template int launch_norm_backward<__nv_bfloat16, float>(const NormBackward&, int, bool, cudaStream_t);
extern template int launch_norm_backward<float, float>(const NormBackward&, int, bool, cudaStream_t);

namespace {

// Adds the teams' sums: a block has 32 columns and 32 lanes of teams, each lane's in their order and then the
// lanes' in theirs; with many teams the blocks of a cluster share them, and their sums meet in the first one's.
constexpr int kSumBlocks = 8;
__global__ void __launch_bounds__(1024) sums_kernel(const __grid_constant__ NormBackward a) {
  __shared__ float part[32][33], whole[32];
  wait_previous();
  const int D = a.io.D, c = blockIdx.x * 32 + threadIdx.x, kind = blockIdx.y;
  const int lanes = 32 * int(gridDim.z), lane = int(blockIdx.z) * 32 + int(threadIdx.y);
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int i = lane; i < a.slots; i += lanes) s += a.part[((long long)i * a.kinds + kind) * D + c];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = 0.f;
  if (threadIdx.y == 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
    whole[threadIdx.x] = s;
  }
  if (gridDim.z > 1) cluster_sync_all();
  if (blockIdx.z == 0 && threadIdx.y == 0 && c < D) {
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&whole[threadIdx.x]));
    for (unsigned i = 1; i < gridDim.z; ++i) s += __uint_as_float(ld_cluster_u32(cluster_addr(mine, i)));
    int k = kind;
    void* out = nullptr;
    for (void* o : {a.dafter, a.dscale, a.dweight})
      if (o && k-- == 0) out = o;
    if (a.io.w_dtype == SDM_F32)
      static_cast<float*>(out)[c] = s;
    else
      static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
  }
  if (gridDim.z > 1) cluster_sync_all();  // the sums outlive their readers
}

// Teams of a group: as many as the card holds at once, and no more than there are rows.
template <int KIND>
int teams_for(int n) {
  return norm_by_width<512, KIND == kStream>(n, [&](auto tpr, auto pieces) {
    constexpr int block = norm_block(tpr);
    return 152 * (sm_threads(KIND, pieces) / block) * (block / int(tpr));
  });
}
int slots_for(long long M, int D, int groups, int parts) {
  const int teams = norm_instance(parts, [&](auto kind) { return teams_for<kind>(D / groups); });
  const long long s = teams / groups < 1 ? 1 : teams / groups;
  return int(s < M ? s : M);
}

int launch_sums(const NormBackward& a, cudaStream_t s) {
  if (!a.kinds) return SDM_OK;
  // More blocks where the columns are few: eight a column tile took 15 us longer at 3 x 1536 columns, and one took 18 us
  // longer at 3 x 100 (4,864 teams).
  const unsigned tiles = unsigned((a.io.D + 31) / 32) * unsigned(a.kinds);
  unsigned blocks = 1;
  while (blocks < kSumBlocks && a.slots > 256 && tiles * blocks * 2 <= 152) blocks *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = blocks;
  attr[1] = after_previous();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((a.io.D + 31) / 32), unsigned(a.kinds), blocks);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.io.M > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, sums_kernel, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_residual_norm_backward_workspace_size(long long M, int D, int groups) {
  if (M < 1 || D < 1 || groups < 1 || D % groups || D / groups > kNormMax) return 0;
  int most = 0;
  for (int parts = 0; parts <= kAny; ++parts) {
    const int s = slots_for(M, D, groups, parts);
    most = s > most ? s : most;
  }
  return size_t(most) * 3 * D * 4;
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
  NormBackward a = {};
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
  auto rows16 = [](const void* p, long long rs) { return !misaligned(p, 15) && rs % 8 == 0; };
  const bool vec = (io.D / io.groups) % 8 == 0 && rows16(io.x, io.x_rs) && rows16(io.gate, io.gate_rs) &&
                   rows16(g.dy, g.dy_rs) && rows16(g.r, g.r_rs) && rows16(g.dr, g.dr_rs) && !misaligned(g.dx, 15) &&
                   !misaligned(g.dgate, 15) && !misaligned(g.dresidual, 15) && !misaligned(io.after, 15) &&
                   !misaligned(io.scale, 15) && !misaligned(io.weight, 15);
  const bool gated = io.gate && io.act == SDM_ACT_SILU;
  const int parts = (g.dy ? kStream : 0) | (io.after ? kAfter : 0) | (gated ? kGate : 0) | (io.scale ? kScale : 0) |
                    (io.gate && !gated ? kAny : 0);
  a.slots = slots_for(io.M, io.D, io.groups, parts);
  const int r = io.x_dtype == SDM_F32   ? launch_norm_backward<float, float>(a, parts, vec, s)
                : io.r_dtype == SDM_F32 ? launch_norm_backward<__nv_bfloat16, float>(a, parts, vec, s)
                                        : launch_norm_backward<__nv_bfloat16, __nv_bfloat16>(a, parts, vec, s);
  return r != SDM_OK ? r : launch_sums(a, s);
}
