// Products on the tcgen05 tensor cores with work in their epilogues: the gated projections, the projections with
// bias, activation and residual, and the two products of either's gradient (sdm_gated.cu, sdm_dense.cu).
//
// One kernel, a persistent pair of CTAs (cta_group::2) that forms 256 x 256 tiles with fp32 accumulators in TMEM,
// double-buffered, TMA feeding a ring of stages (the roles of the projection kernel in sdm_project.cu, with eight
// epilogue warps: with four, kSlope's elementwise work was longer than its products):
//   kForward     the pair's two halves of the column tile are 128 columns of Wg and the same 128 of Wu, so one
//                thread of the epilogue holds g and u of an element and h leaves the chip once: neither g nor u is ever
//                written.
//   kSlope       the same product again in the backward pass (g and u were not kept: 4F bytes a token less to hold
//                between the passes, for a third of the backward's flops); its epilogue takes dh and leaves dg and
//                du, rounded to bf16 for the two products that follow.
//   kGrads       those two in one launch, so that their tiles share the card's last round: dx = dz w, where w's rows
//                are the reduction and its tile is read MN-major, and dw = dz^T x, where the tokens are and both
//                operands are MN-major (dz = [dg | du] of the gated projections).
//   kDense       z = x w^T on plain column tiles; y = residual + act(z + bias).
//   kDenseSlope  the same product in the backward pass: dz = dy act'(z + bias), rounded to bf16 for kGrads.
// No operand is transposed in memory: TMA boxes of 64 x 64 in the 128-byte swizzle serve as either major, and only
// the descriptors differ.  Sums are fp32.  What an epilogue takes and leaves goes through patches of 32 rows x 64 columns by TMA.
#pragma once

#include "sdm_layers.cuh"
#include "sdm_tcgen05.cuh"

namespace sdm {
namespace {

enum Mode { kForward = 0, kSlope = 1, kGrads = 2, kDense = 3, kDenseSlope = 4 };
enum Grads { kBoth = 0, kInput = 1, kWeight = 2 };  // what a kGrads launch computes

constexpr int kHalf = 128;                       // rows (and columns) of a tile each CTA stages
constexpr int kOperand = kHalf * kTileK * 2;     // 16 KB
constexpr int kStage = 2 * kOperand;
constexpr int kEpilogueWarps = 8;                // two for each quarter of the tile's rows
constexpr int kRoles = 64 + 32 * kEpilogueWarps; // copy warp, MMA warp, epilogue warps
constexpr int kPatch = 32 * 64 * 2;               // 32 rows x 64 columns of bf16: a warp's output
// Shared memory: a ring of stages, then patches through which the epilogue warps load and store.
template <int MODE>
struct Layout {
  static constexpr int patches = MODE == kGrads ? 0 : MODE == kForward ? 1 : 2;  // of each warp
  static constexpr int stages = patches == 2 ? 5 : 6;
  static constexpr int bars = 2 * stages + 5 + kEpilogueWarps;  // full[], empty[], acc_full[2],
                                                                // acc_empty[2], drain, patch[]
  static constexpr int off_patch = stages * kStage;
  static constexpr int off_bars = off_patch + patches * kEpilogueWarps * kPatch;
  static constexpr int bytes = off_bars + 512 + 1024 /* alignment slack */;
};
constexpr uint32_t kColumns = 512;
constexpr int kRowGroup = 32;                    // row tiles of a group of the tile order, where nothing else is said

// One product: its output [rows, cols], its tiles, and the cut of its reduction (K steps of 64).
struct Product {
  int rows, cols;
  int row_tiles, col_tiles, splits;
  int kblocks, per_split;
  int group;               // row tiles of a group of the tile order
  bool a_mn;               // kGrads: A read MN-major (dw)
  __nv_bfloat16* out;      // kGrads: dx or dw
  float* partial;          // [splits][rows][cols] where splits > 1
  __host__ __device__ int units() const { return row_tiles * col_tiles * splits; }
};
struct ProductArgs {
  Product p[2];            // kGrads: both, the one of longer units first; otherwise the first
  int act;
  const __nv_bfloat16* bias;   // kDense, kDenseSlope: or null
  const __nv_bfloat16* extra;  // kDense: the residual or null; kDenseSlope: dy
  float* sums;                 // kDenseSlope: [rows / 32][cols], dz summed over 32 rows each, or null
  int* dev_err;
};

// D fp32, A and B bf16, M 256, N 256; bits 15 and 16: A, B MN-major.
constexpr uint32_t idesc(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t(256 >> 3) << 17) | (uint32_t(256 >> 4) << 24);
}

// MN-major operand of boxes of 64 (MN) x 64 (K): a box is 64 K rows of 128 bytes, 8-row atoms of
// 1,024 bytes stacked along K (stride byte offset), the next 64 along MN one box further (leading
// byte offset 8,192).  A K step of 16 is two atoms: 2,048 bytes.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(8192 >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate,
                                     uint32_t id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(accumulate), "r"(id)
      : "memory");
}

// Phi(g) of the exact gelu, g Phi(g), and e = exp(-g^2 / 2), which its slope needs too:
// Phi(-|g|) = erfc(x) / 2 with x = |g| / sqrt(2) = e t p(t) / 2, t = 1 / (1 + 0.4 x), where p is the
// polynomial of degree 8 nearest to erfc(x) exp(x^2) / t on 0 < t <= 1 in relative error (1.3e-7;
// 5e-7 with its roundings), by weighted least squares on Chebyshev points, the weights moved until the
// error was level.  The tail keeps its relative precision, and erfc and exp share an exponential.
__device__ __forceinline__ float gelu_cdf(float g, float& e) {
  e = exp2_fast(-0.5f * kLog2e * g * g);
  const float t = rcp_fast(fmaf(fabsf(g), 0.4f * 0.70710678118654752f, 1.0f));
  float p = fmaf(t, 0.05026422068476677f, -0.18291062116622925f);
  p = fmaf(t, p, 0.16910173f);
  p = fmaf(t, p, -0.005622821860015392f);
  p = fmaf(t, p, 0.1414395123720169f);
  p = fmaf(t, p, 0.16853958368301392f);
  p = fmaf(t, p, 0.20784306526184082f);
  p = fmaf(t, p, 0.22566957771778107f);
  p = fmaf(t, p, 0.22567586600780487f);
  const float q = 0.5f * e * (t * p);
  return g > 0.0f ? 1.0f - q : q;
}
template <int ACT>
__device__ __forceinline__ float gate(float g) {
  float e;
  return ACT == SDM_ACT_SILU ? silu(g) : g * gelu_cdf(g, e);
}
// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void gate_slope(float g, float& a, float& s) {
  if (ACT == SDM_ACT_SILU) {
    const float p = sigmoid(g);
    a = g * p;
    s = fmaf(a, 1.0f - p, p);
  } else {
    float e;
    const float p = gelu_cdf(g, e);
    a = g * p;
    s = fmaf(g * 0.39894228040143268f, e, p);
  }
}

// Work unit -> product, row tile, column tile, split: groups of row tiles, row tiles
// fastest, so that units running at once share a few rows of A and a few column tiles of B in L2.
struct Unit {
  int which, row, col, k_lo, k_hi, split;
};
template <int MODE, int KIND>
__device__ __forceinline__ Unit unit_at(int u, const ProductArgs& a) {
  Unit r;
  r.which = 0;
  if (MODE == kGrads && KIND == kBoth && u >= a.p[0].units()) {
    u -= a.p[0].units();
    r.which = 1;
  }
  const Product& p = a.p[r.which];
  const int tiles = p.row_tiles * p.col_tiles;
  r.split = u / tiles;
  u -= r.split * tiles;
  const int g = u / (p.group * p.col_tiles), w = u - g * p.group * p.col_tiles;
  const int gm = min(p.group, p.row_tiles - g * p.group);
  r.col = w / gm;
  r.row = g * p.group + (w - r.col * gm);
  r.k_lo = r.split * p.per_split;
  r.k_hi = min(p.kblocks, r.k_lo + p.per_split);
  return r;
}

// 16-byte piece j of row r of a patch in the 128-byte swizzle that its copies use.
__device__ __forceinline__ uint32_t patch_at(int r, int j) { return uint32_t(r * 128 + ((j ^ (r & 7)) << 4)); }
__device__ __forceinline__ uint4 patch_load(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p));
  return v;
}
__device__ __forceinline__ void patch_store(uint32_t p, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void patch_copy_out(const CUtensorMap* map, int x, int y, uint32_t p) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(p)
               : "memory");
}
__device__ __forceinline__ void copies_out_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_out_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void copies_out_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// h, or dg and du, of a warp's 32 rows x 64 columns: from TMEM (gate and up columns) through
// registers into the warp's patches.  kSlope's first patch holds dh on entry and dg on exit.
template <int MODE, int ACT>
__device__ __forceinline__ void gate_patch(uint32_t tgate, uint32_t tup, uint32_t patch, int lane) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t g[16], u[16];
    tmem_load16(tgate + uint32_t(c), g);
    tmem_load16(tup + uint32_t(c), u);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t at = patch + patch_at(lane, c / 8 + j);
      float o[8];
      if constexpr (MODE == kForward) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = gate<ACT>(__uint_as_float(g[8 * j + i])) * __uint_as_float(u[8 * j + i]);
        patch_store(at, Piece<__nv_bfloat16>::pack(o));
      } else {
        float d[8], o2[8];
        Piece<__nv_bfloat16>::load(patch_load(at), d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v, s;
          gate_slope<ACT>(__uint_as_float(g[8 * j + i]), v, s);
          o[i] = d[i] * __uint_as_float(u[8 * j + i]) * s;
          o2[i] = d[i] * v;
        }
        patch_store(at, Piece<__nv_bfloat16>::pack(o));
        patch_store(at + kPatch, Piece<__nv_bfloat16>::pack(o2));
      }
    }
  }
}

template <int ACT>
__device__ __forceinline__ float dense_act(float z) {
  if constexpr (ACT == SDM_ACT_NONE) return z;
  else return gate<ACT>(z);
}
// What leaves a dense product's epilogue for eight columns of z: residual + act(z + bias) or dy act'(z + bias).
// `extra` holds the residual or dy.
template <int MODE, int ACT>
__device__ __forceinline__ uint4 dense_piece(float (&z)[8], const __nv_bfloat16* bias, bool has_extra, const uint4& extra) {
  float e[8];
  if (bias) {
    Piece<__nv_bfloat16>::load(__ldg(reinterpret_cast<const uint4*>(bias)), e);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += e[i];
  }
  if (has_extra) Piece<__nv_bfloat16>::load(extra, e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (MODE == kDense) {
      z[i] = dense_act<ACT>(z[i]);
      if (has_extra) z[i] += e[i];
    } else {
      float v, s;
      gate_slope<ACT>(z[i], v, s);
      z[i] = e[i] * s;
    }
  }
  return Piece<__nv_bfloat16>::pack(z);
}
// A warp's 32 rows x 64 columns of a dense product: from TMEM through registers into its patch, which holds the
// residual or dy on entry.  bias: at the patch's first column; cols: columns inside the matrix.
template <int MODE, int ACT>
__device__ __forceinline__ void dense_patch(uint32_t taddr, uint32_t patch, int lane, const __nv_bfloat16* bias, bool has_extra,
                                            int cols) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t r[16];
    tmem_load16(taddr + uint32_t(c), r);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = c + 8 * j;
      const uint32_t at = patch + patch_at(lane, col / 8);
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = __uint_as_float(r[8 * j + i]);
      patch_store(at, dense_piece<MODE, ACT>(z, bias && col < cols ? bias + col : nullptr, has_extra,
                                             has_extra ? patch_load(at) : make_uint4(0, 0, 0, 0)));
    }
  }
}

// Sums over a patch's rows, two columns a lane; rows past the matrix are 0 (dy is).
__device__ __forceinline__ void dense_sums(uint32_t patch, int lane, float* out, int cols) {
  float s0 = 0.f, s1 = 0.f;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(patch + patch_at(r, lane / 4) + uint32_t(lane % 4 * 4)));
    s0 += __uint_as_float(w << 16);
    s1 += __uint_as_float(w & 0xFFFF0000u);
  }
  if (2 * lane < cols) *reinterpret_cast<float2*>(out + 2 * lane) = make_float2(s0, s1);
}

// Sums of a warp's 32 rows x 128 columns, straight to memory: dx or dw, or partial sums.
__device__ __forceinline__ void store_sums(const Product& a, const Unit& un, int m, int n0, uint32_t taddr) {
#pragma unroll 1
  for (int c = 0; c < kHalf; c += 32) {
    uint32_t r[32];
    tmem_load32(taddr + uint32_t(c), r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + c + 8 * j;
      if (m >= a.rows || n >= a.cols) break;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(r[8 * j + i]);
      if (a.splits > 1) {
        float* p = a.partial + (size_t(un.split) * a.rows + m) * a.cols + n;
        *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(o[4], o[5], o[6], o[7]);
      } else {
        *reinterpret_cast<uint4*>(a.out + size_t(m) * a.cols + n) = Piece<__nv_bfloat16>::pack(o);
      }
    }
    __syncwarp();  // tcgen05.ld takes the whole warp
  }
}

// Tensor maps of a launch: the operands of each product (kForward, kSlope: B[1] is the rank-1 CTA's,
// Wu), and what the epilogue moves in patches: dh, dy or the residual in; h, dg and du, y or dz out.
struct Maps {
  CUtensorMap A[2], B[2], in, out, out2;
};

// KIND: the activation, or of kGrads the products (known where there is one, so that the one thread
// that issues MMAs has nothing to choose: 2 % of the whole gradient).
// Every wait is bounded; a wait that runs out stops both CTAs, which drain the copies and MMAs in
// flight, free TMEM and report SDM_DEV_TIMEOUT.
template <int MODE, int KIND>
__global__ void __launch_bounds__(kRoles, 1)
    product_kernel(const __grid_constant__ Maps tm, const __grid_constant__ ProductArgs a) {
  using Lay = Layout<MODE>;
  constexpr int kStages = Lay::stages;
  constexpr bool kGate = MODE == kForward || MODE == kSlope;
  constexpr bool kPlain = MODE == kDense || MODE == kDenseSlope;
  constexpr bool kBMN = MODE == kGrads;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (ring - raw) + Lay::off_bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Lay::bars);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued = tmem_slot + 2;  // copies issued per stage, read by the leader after a stop
  const int FULL = 0, EMPTY = kStages, ACC_FULL = 2 * kStages, ACC_EMPTY = 2 * kStages + 2,
            DRAIN = 2 * kStages + 4, PATCH = 2 * kStages + 5;
  auto bar = [&](int i) { return smem_u32(bars + i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const uint32_t peer_stop = cluster_addr(smem_u32(const_cast<int*>(stop)), rank ^ 1u);
  const int cid = blockIdx.x / 2, ncl = gridDim.x / 2;
  const int units = a.p[0].units() + (MODE == kGrads && KIND == kBoth ? a.p[1].units() : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(FULL + s), 1);   // the leader's expect_tx; both CTAs' bytes
      mbar_init(bar(EMPTY + s), 1);  // the leader's commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(ACC_FULL + i), 1);
      mbar_init(bar(ACC_EMPTY + i), 2 * kEpilogueWarps);  // both CTAs' epilogue warps
    }
    mbar_init(bar(DRAIN), 1);
    for (int i = 0; i < kEpilogueWarps; ++i) mbar_init(bar(PATCH + i), 1);
    *stop = 0;
    for (int s = 0; s < kStages; ++s) issued[s] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm.A[0])) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm.B[0])) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  allow_next();
  if (MODE == kGrads) wait_previous();  // kSlope's dg and du

  if (warp == 0) {
    if (lane == 0) {
      // ---- copies (both CTAs) ----
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int u = cid; ok && u < units; u += ncl) {
        const Unit un = unit_at<MODE, KIND>(u, a);
        const CUtensorMap* mapA = &tm.A[un.which];
        const CUtensorMap* mapB = &tm.B[kGate ? int(rank) : un.which];
        const bool a_mn = MODE == kGrads && (KIND == kBoth ? a.p[un.which].a_mn : KIND == kWeight);
        const int m0 = (un.row * 2 + int(rank)) * kHalf;
        const int n0 = kGate ? un.col * kHalf : un.col * 2 * kHalf + int(rank) * kHalf;
        for (int kb = un.k_lo; kb < un.k_hi; ++kb) {
          if (!mbar_wait_cluster(bar(EMPTY + stage), phase ^ 1u, stop, peer_stop, kWaitNs)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + uint32_t(stage) * kStage, sb = sa + kOperand;
          const uint32_t full = cluster_addr(bar(FULL + stage), 0);
          if (leader) mbar_expect_tx(bar(FULL + stage), 2 * kStage);
          if (a_mn) {
            tma_load_2d_pair(sa, mapA, m0, kb * kTileK, full);
            tma_load_2d_pair(sa + kOperand / 2, mapA, m0 + kHalf / 2, kb * kTileK, full);
          } else {
            tma_load_2d_pair(sa, mapA, kb * kTileK, m0, full);
          }
          if (kBMN) {
            tma_load_2d_pair(sb, mapB, n0, kb * kTileK, full);
            tma_load_2d_pair(sb + kOperand / 2, mapB, n0 + kHalf / 2, kb * kTileK, full);
          } else {
            tma_load_2d_pair(sb, mapB, kb * kTileK, n0, full);
          }
          issued[stage] = issued[stage] + 1u;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---- MMAs (leader only) ----
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;
      for (int u = cid; ok && u < units; u += ncl, ++it) {
        const Unit un = unit_at<MODE, KIND>(u, a);
        const bool a_mn = MODE == kGrads && (KIND == kBoth ? a.p[un.which].a_mn : KIND == kWeight);
        const uint32_t id = a_mn ? idesc(true, kBMN) : idesc(false, kBMN);
        const int acc = it & 1;
        const uint32_t acc_par = uint32_t(it >> 1) & 1u;
        if (!mbar_wait_cluster(bar(ACC_EMPTY + acc), acc_par ^ 1u, stop, peer_stop, kWaitNs)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + uint32_t(acc * 256);
        for (int kb = un.k_lo; kb < un.k_hi; ++kb) {
          if (!mbar_wait_cluster(bar(FULL + stage), phase, stop, peer_stop, kWaitNs)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = ring + uint32_t(stage) * kStage, sb = sa + kOperand;
#pragma unroll
          for (int kk = 0; kk < kTileK / 16; ++kk)
            mma2(d, a_mn ? mn_desc(sa + kk * 2048) : sw128_desc(sa + kk * 32),
                 kBMN ? mn_desc(sb + kk * 2048) : sw128_desc(sb + kk * 32), kb > un.k_lo || kk > 0, id);
          mma2_commit_both(bar(EMPTY + stage));
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) mma2_commit_both(bar(ACC_FULL + acc));
      }
      mma2_commit_local(bar(DRAIN));
      mbar_wait_teardown(bar(DRAIN), 0);
    }
  } else {
    // ---- epilogue (both CTAs): warp w reads TMEM lanes 32 * (w % 4) .. + 31, half of the columns ----
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t patch = ring + Lay::off_patch + uint32_t((warp - 2) * Lay::patches * kPatch);
    const uint32_t patch_bar = bar(PATCH + warp - 2);
    uint32_t patch_loads = 0;  // loads of the patches asked for, and how many of them were awaited
    uint32_t patch_waits = 0;
    int it = 0;
    for (int u = cid; u < units; u += ncl, ++it) {
      const int acc = it & 1;
      const uint32_t acc_par = uint32_t(it >> 1) & 1u;
      const Unit un = unit_at<MODE, KIND>(u, a);
      const int m0 = (un.row * 2 + int(rank)) * kHalf + quad * 32;
      const int f0 = kPlain ? un.col * 2 * kHalf + half * kHalf : un.col * kHalf + half * 64;
      // A patch outside the matrix is neither loaded nor stored; one across its edge is cut there.
      const bool whole = !kPlain || a.p[0].splits == 1;  // otherwise sums leave, for join_dense_kernel
      const bool inside = (kGate || kPlain) && whole && m0 < a.p[0].rows && f0 < a.p[0].cols;
      const bool inside2 = kPlain && inside && f0 + 64 < a.p[0].cols;
      const bool loads = MODE == kSlope || (kPlain && a.extra);
      if ((kGate || kPlain) && lane == 0) copies_out_read();  // the patches' last copies have read them
      if (loads && inside) {
        if (lane == 0) {
          mbar_expect_tx(patch_bar, inside2 ? 2 * kPatch : kPatch);
          tma_load_2d(patch, &tm.in, f0, m0, patch_bar);
          if (inside2) tma_load_2d(patch + kPatch, &tm.in, f0 + 64, m0, patch_bar);
        }
        ++patch_loads;
      }
      __syncwarp();
      if (!__all_sync(0xFFFFFFFFu,
                      mbar_wait_cluster(bar(ACC_FULL + acc), acc_par, stop, peer_stop, kWaitNs)))
        break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + (uint32_t(quad * 32) << 16) + uint32_t(acc * 256);
      if constexpr (kGate) {
        if (inside) {
          if (MODE == kSlope) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(patch_bar, patch_waits & 1u, stop, peer_stop, kWaitNs)))
              break;
            ++patch_waits;
          }
          gate_patch<MODE, KIND>(taddr + uint32_t(half * 64), taddr + uint32_t(kHalf + half * 64), patch, lane);
          fence_async_proxy();
        }
      } else if constexpr (kPlain) {
        if (inside) {
          if (loads) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(patch_bar, patch_waits & 1u, stop, peer_stop, kWaitNs)))
              break;
            ++patch_waits;
          }
          const __nv_bfloat16* bias = a.bias ? a.bias + f0 : nullptr;
          const uint32_t from = taddr + uint32_t(half * kHalf);
          dense_patch<MODE, KIND>(from, patch, lane, bias, loads, a.p[0].cols - f0);
          if (inside2)
            dense_patch<MODE, KIND>(from + 64, patch + kPatch, lane, bias ? bias + 64 : nullptr, loads,
                                    a.p[0].cols - f0 - 64);
          fence_async_proxy();
          if (MODE == kDenseSlope && a.sums) {
            __syncwarp();
            dense_sums(patch, lane, a.sums + size_t(m0 / 32) * a.p[0].cols + f0, a.p[0].cols - f0);
            if (inside2)
              dense_sums(patch + kPatch, lane, a.sums + size_t(m0 / 32) * a.p[0].cols + f0 + 64, a.p[0].cols - f0 - 64);
          }
        } else if (!whole) {
          store_sums(a.p[0], un, m0 + lane, f0, taddr + uint32_t(half * kHalf));
        }
      } else {
        store_sums(a.p[un.which], un, m0 + lane, un.col * 2 * kHalf + half * kHalf, taddr + uint32_t(half * kHalf));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(cluster_addr(bar(ACC_EMPTY + acc), 0));
        if (inside) {
          patch_copy_out(&tm.out, f0, m0, patch);
          if (MODE == kSlope) patch_copy_out(&tm.out2, f0, m0, patch + kPatch);
          if (inside2) patch_copy_out(&tm.out, f0 + 64, m0, patch + kPatch);
        }
        if (kGate || kPlain) copies_out_commit();
      }
    }
    if ((kGate || kPlain) && lane == 0) {
      copies_out_done();
      if (patch_waits != patch_loads) mbar_wait_teardown(patch_bar, patch_waits & 1u);
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kColumns)
                 : "memory");
  if (leader && warp == 0 && lane == 0 && *stop) {
    // After a stop, every copy either CTA issued lands before the pair's shared memory goes away:
    // per stage the two issued the same number of copies or one more than the other; the leader
    // arms a phase only its peer issued with the peer's bytes, counts the peer's missing bytes of
    // a phase only it issued as done, and waits for the last phase of each stage.
    const uint32_t peer_issued = cluster_addr(smem_u32(const_cast<uint32_t*>(issued)), 1u);
    for (int s = 0; s < kStages; ++s) {
      const uint32_t lc = issued[s], pc = ld_cluster_u32(peer_issued + 4u * uint32_t(s));
      if (pc == lc + 1u) {
        mbar_expect_tx(bar(FULL + s), kStage);
        mbar_wait_teardown(bar(FULL + s), lc & 1u);
      } else if (lc == pc + 1u) {
        mbar_complete_tx(bar(FULL + s), kStage);
        mbar_wait_teardown(bar(FULL + s), (lc - 1u) & 1u);
      } else if (lc == pc && lc > 0u) {
        mbar_wait_teardown(bar(FULL + s), (lc - 1u) & 1u);
      }
    }
  }
  if (threadIdx.x == 0 && *stop && a.dev_err) atomicOr(a.dev_err, SDM_DEV_TIMEOUT);
  cluster_sync_all();  // the peer's shared memory outlives the leader's drain
}

// Sums the splits' partial results of the products that have any, in their order, and rounds once.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ ProductArgs a, unsigned first_blocks) {
  wait_previous();
  const Product& p = a.p[blockIdx.x >= first_blocks];
  const unsigned block = blockIdx.x >= first_blocks ? blockIdx.x - first_blocks : blockIdx.x;
  const size_t n = size_t(p.rows) * p.cols, i = (size_t(block) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4* q = reinterpret_cast<const float4*>(p.partial + size_t(s) * n + i);
    const float4 v = __ldcs(q), w = __ldcs(q + 1);
    o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
    o[4] += w.x, o[5] += w.y, o[6] += w.z, o[7] += w.w;
  }
  *reinterpret_cast<uint4*>(p.out + i) = Piece<__nv_bfloat16>::pack(o);
}

// The same for a dense product, with its epilogue.
template <int MODE, int ACT>
__global__ void __launch_bounds__(256) join_dense_kernel(const __grid_constant__ ProductArgs a) {
  wait_previous();
  const Product& p = a.p[0];
  const size_t n = size_t(p.rows) * p.cols, i = (size_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  uint4 extra = make_uint4(0, 0, 0, 0);
  if (a.extra) extra = *reinterpret_cast<const uint4*>(a.extra + i);
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float4* q = reinterpret_cast<const float4*>(p.partial + size_t(s) * n + i);
    const float4 v = __ldcs(q), w = __ldcs(q + 1);
    o[0] += v.x, o[1] += v.y, o[2] += v.z, o[3] += v.w;
    o[4] += w.x, o[5] += w.y, o[6] += w.z, o[7] += w.w;
  }
  *reinterpret_cast<uint4*>(p.out + i) =
      dense_piece<MODE, ACT>(o, a.bias ? a.bias + i % p.cols : nullptr, a.extra != nullptr, extra);
}

// ---- few tokens: weights streamed past mma.sync (the kernels are in sdm_gated.cu and sdm_dense.cu) ----

constexpr int kFewTokens = 16;

__device__ __forceinline__ uint4 load_stream(const void* p) {  // read once: past L1
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p));
  return v;
}
__device__ __forceinline__ void mma16n8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

constexpr int kPairs = 76;  // pairs of SMs

Product product(int rows, int cols, int tile_cols, long long reduction) {
  Product p = {};
  p.rows = rows;
  p.cols = cols;
  p.row_tiles = ceil_div(rows, 2 * kHalf);
  p.col_tiles = ceil_div(cols, tile_cols);
  p.kblocks = p.per_split = ceil_div(reduction, kTileK);
  p.splits = 1;
  p.group = kRowGroup;
  return p;
}

void cut(Product& p, int splits) {
  p.per_split = ceil_div(p.kblocks, splits);
  p.splits = ceil_div(p.kblocks, p.per_split);  // none of them empty
}

// K steps of the busiest pair, the first, where units are dealt out in turn, those of product a (the
// longer) before those of b.  A unit costs about 8 steps more for its start and its epilogue.
double busiest(const Product& a, const Product& b) {
  const long long na = a.units(), nb = b.units();
  const double ra = double((na + kPairs - 1) / kPairs);
  const long long left = na + nb - (long long)ra * kPairs;
  return ra * (a.per_split + 8) + (left > 0 ? double((left + kPairs - 1) / kPairs) * (b.per_split + 8) : 0.0);
}
// Moving a product's partials twice, and a launch, in K steps (512 clocks of a pair; HBM moves about
// 1.8 MB in one).
double joining(const Product& p) {
  return p.splits > 1 ? double(p.rows) * p.cols * (8.0 * p.splits + 2.0) / 1.8e6 + 5 : 0.0;
}

// With eight rounds of tiles or more the last one's loss is small: neither are reductions split then,
// nor are the products put in one launch.
bool one_launch(const Product (&p)[2]) {
  return (long long)p[0].row_tiles * p[0].col_tiles + (long long)p[1].row_tiles * p[1].col_tiles < 8 * kPairs;
}

// The two products of the gradient, dx and dw, the one of longer units first.  With few tiles
// their reductions are split so that every pair of SMs has its share: the cut of least time among
// up to 8 splits of each.
void plan_grads(int M, int D, int N, Product (&p)[2]) {
  Product x = product(M, D, 2 * kHalf, N), w = product(N, D, 2 * kHalf, M);
  w.a_mn = true;
  Product best[2] = {x, w};
  double least = -1;
  const int most = one_launch(best) ? 8 : 1;
  for (int i = 1; i <= most; ++i)
    for (int j = 1; j <= most; ++j) {
      cut(x, i);
      cut(w, j);
      const bool swap = w.per_split > x.per_split;
      const double t = (swap ? busiest(w, x) : busiest(x, w)) + joining(x) + joining(w);
      if (least < 0 || t < least) {
        least = t;
        best[0] = swap ? w : x;
        best[1] = swap ? x : w;
      }
    }
  p[0] = best[0];
  p[1] = best[1];
}

template <int MODE, int KIND>
int launch_mode(const Maps& tm, const ProductArgs& a, cudaStream_t s) {
  const long long units = (long long)a.p[0].row_tiles * a.p[0].col_tiles * a.p[0].splits +
                          (MODE == kGrads && KIND == kBoth ? (long long)a.p[1].row_tiles * a.p[1].col_tiles * a.p[1].splits : 0);
  if (units > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  auto fn = product_kernel<MODE, KIND>;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = after_previous();
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRoles);
  cfg.dynamicSmemBytes = Layout<MODE>::bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Pairs that can be resident at once: a larger persistent grid would run in two waves.
  static PerDevice resident;
  long long pairs = resident.get([&] {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<MODE>::bytes) != cudaSuccess)
      return -1;
    const int most = sm_count() / 2;
    cfg.gridDim = dim3(unsigned(most > 0 ? most * 2 : 2));
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, fn, &cfg) != cudaSuccess || active <= 0) return -1;
    return active < most ? active : most;
  });
  if (pairs <= 0) return SDM_ECUDA;
  if (units < pairs) pairs = units;
  cfg.gridDim = dim3(unsigned(pairs * 2));
  if (MODE == kGrads) cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, fn, tm, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

int launch_join(const ProductArgs& a, cudaStream_t s) {
  unsigned blocks[2];
  for (int i = 0; i < 2; ++i)
    blocks[i] = a.p[i].splits > 1 ? unsigned((size_t(a.p[i].rows) * a.p[i].cols / 8 + 255) / 256) : 0;
  if (blocks[0] + blocks[1] == 0) return SDM_OK;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks[0] + blocks[1]);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_kernel, a, blocks[0]) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t partial_bytes(const Product& p) {
  return p.splits > 1 ? round256(size_t(p.splits) * p.rows * p.cols * 4) : 0;
}


// dx = dz w and dw = dz^T x for dz [M, N], w [N, D], x [M, D]; `partial`: the sums of split products.
int launch_grads(const __nv_bfloat16* dz, const void* x, const void* w, int M, int D, int N, void* dx, void* dw,
                 uint8_t* partial, int* dev_err, cudaStream_t s) {
  ProductArgs a = {};
  plan_grads(M, D, N, a.p);
  const int ix = a.p[0].a_mn ? 1 : 0, iw = 1 - ix;  // dx's place, dw's
  Maps tg = {};
  if (!bf16_tile_map(&tg.A[ix], dz, M, N, kHalf) || !bf16_tile_map(&tg.B[ix], w, N, D, kTileK) ||
      !bf16_tile_map(&tg.A[iw], dz, M, N, kTileK) || !bf16_tile_map(&tg.B[iw], x, M, D, kTileK))
    return SDM_ECUDA;
  a.dev_err = dev_err;
  a.p[0].partial = reinterpret_cast<float*>(partial);
  a.p[1].partial = reinterpret_cast<float*>(partial + partial_bytes(a.p[0]));
  a.p[ix].out = static_cast<__nv_bfloat16*>(dx);
  a.p[iw].out = static_cast<__nv_bfloat16*>(dw);
  if (!one_launch(a.p)) {
    auto alone = [&](int i, ProductArgs& one, Maps& maps) {
      one = a;
      one.p[0] = a.p[i];
      maps = tg;
      maps.A[0] = tg.A[i];
      maps.B[0] = tg.B[i];
    };
    ProductArgs one;
    Maps maps;
    alone(ix, one, maps);
    const int st = launch_mode<kGrads, kInput>(maps, one, s);
    if (st != SDM_OK) return st;
    alone(iw, one, maps);
    return launch_mode<kGrads, kWeight>(maps, one, s);
  }
  const int st = launch_mode<kGrads, kBoth>(tg, a, s);
  return st != SDM_OK ? st : launch_join(a, s);
}

}  // namespace
}  // namespace sdm
