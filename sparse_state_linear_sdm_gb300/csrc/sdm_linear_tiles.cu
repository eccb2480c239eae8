// Linear attention over prompts in chunks of 128 tokens on the tcgen05 tensor cores (bf16, up to 128 columns).
//
// With A_ij the product of the decays of tokens j+1 .. i of a chunk, S the state in front of it and G the products from its start:
//
//   o_i = scale (sum_{j<=i} A_ij (q_i k_j) v_j  +  G_i q_i S)
//   S'  = G_last S + sum_j k_j (A_last,j v_j)^T
//
// Four products a chunk: q k^T, q S, (A q k^T) v and k^T (A v).  A CTA takes a sequence's head, its state in
// registers (fp32, 64 a thread), and walks its chunks; every product has its accumulator in TMEM (128 columns each,
// all 512 together).  Warps by role: TMA and decays; MMAs; eight that turn q k^T into the masked bf16 products and
// write o; eight that weight v and update the state.  q, k and v come through a ring of four 32 KB slots, in
// the order of their use, so that the slot of q takes the next k, and so on.
//
// What is rounded to bf16: the masked products and the state as q reads it, as an MMA takes them (each half a unit, as o
// itself).  The state is not: A v is cut into three bf16 parts whose products are summed in fp32 (two parts
// leave 3e-6 of the state, three 1e-8), which costs two more MMAs of six a chunk and no byte.
// The A_ij of a row are formed by one product after the other from the diagonal on, so a decay of 0 leaves 0 before it
// and no difference of sums is taken; G and A_last,j come from sums of g in 64 bits.
#include "sdm_linear.cuh"
#include "sdm_tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kChunk = 128;
constexpr int kSlot = 32768;             // 128 tokens of 128 columns: two boxes of 64 columns
constexpr int kBox = kChunk * 128;       // bytes of a box
constexpr int kSlots = 4;
constexpr int kSlice = 16;               // tokens of a weighted slice of v: one K step
constexpr int kTileThreads = 32 * 18;
constexpr int kMaskWarp = 2, kStateWarp = 10;  // first warps of the two groups of eight

enum Bar {
  kFull = 0, kEmpty = 4,          // slots
  kScoreFull = 8, kScoreEmpty,    // q k^T
  kMaskFull, kMaskEmpty,          // the masked products in shared memory
  kOutFull, kOutEmpty,            // both accumulators of o
  kStateFull, kStateEmpty,        // the state as q reads it
  kPartFull, kPartEmpty = kPartFull + 2,  // weighted slices
  kSumFull = kPartEmpty + 2, kSumEmpty,   // k^T (A v)
  kDecayFull, kDecayEmpty = kDecayFull + 2,
  kCut = kDecayEmpty + 2,         // tokens past the end cleared
  kDrain, kBars
};

struct Decays {  // of a chunk
  float each[kChunk];  // e^g
  float from[kChunk];  // products from the chunk's start up to each token
  float to[kChunk];    // products after each token up to the chunk's end; 0 past the sequence's
  float all, pad[3];
};

template <int DK, int DV>
struct Tiles {
  static constexpr int part = DV / 64 * kSlice * 128;  // one of three parts of a slice
  static constexpr int off_state = kSlots * kSlot;
  static constexpr int off_mask = off_state + DK * DV * 2;
  static constexpr int off_parts = off_mask + 2 * kBox;
  static constexpr int off_decays = off_parts + 2 * 3 * part;
  static constexpr int off_bars = off_decays + 2 * int(sizeof(Decays));
  static constexpr int bytes = off_bars + 512 + 1024 /* alignment slack */;
};

constexpr uint32_t kScore = 0, kOutState = 128, kOutChunk = 256, kSum = 384;  // TMEM columns

struct TileMaps {
  CUtensorMap q, k, v;
};

// D fp32, A and B bf16, M 128; bits 15 and 16: A, B MN-major.
constexpr uint32_t tile_idesc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t(n >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
// MN-major operand in boxes of 64 columns, `box` bytes apart; a K step of 16 rows is 2,048 bytes.
__device__ __forceinline__ uint64_t mn_box_desc(uint32_t saddr, uint32_t box) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(box >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void mma1(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %3, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(accumulate), "r"(id)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return uint32_t(row * 128 + ((piece ^ (row & 7)) << 4)); }
__device__ __forceinline__ uint4 shared_load(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void shared_store(uint32_t p, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 2^x, at most the largest float: times a state of 0 it is 0.
__device__ __forceinline__ float finite_exp2(float x) {
  const float y = exp2f(x);
  return y > 3.402823466e38f ? 3.402823466e38f : y;
}

// Every wait is bounded; one that runs out stops the CTA, which waits for the copies and MMAs in flight, frees TMEM and
// reports SDM_DEV_TIMEOUT.
template <int DK, int DV, int PASS>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ TileMaps tm, const __grid_constant__ LinearArgs a) {
  typedef Tiles<DK, DV> L;
  constexpr int kBoxesK = DK / 64, kBoxesV = DV / 64;
  constexpr int kLoads = PASS == kReduce ? 2 : 3;  // slots a chunk takes
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::off_bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued = tmem_slot + 2;
  Decays* decays = reinterpret_cast<Decays*>(smem + L::off_decays);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const sdm_linear_args& io = a.io;

  if (PASS == kReduce) allow_next();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      int n = 1;
      if (i == kScoreEmpty || i == kMaskFull || i == kOutEmpty || i == kStateFull || i == kPartFull || i == kPartFull + 1 ||
          i == kSumEmpty || i == kCut)
        n = 8;  // the warps of a group
      if (i == kDecayEmpty || i == kDecayEmpty + 1) n = PASS == kReduce ? 8 : 16;
      mbar_init(bar(i), uint32_t(n));
    }
    *stop = 0;
    for (int i = 0; i < kSlots; ++i) issued[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The masked products' blocks above the diagonal stay 0.
  if (PASS != kReduce) {
    for (uint32_t i = threadIdx.x * 16; i < 2 * kBox; i += kTileThreads * 16)
      *reinterpret_cast<uint4*>(smem + L::off_mask + i) = make_uint4(0, 0, 0, 0);
    async_proxy_fence();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Place p = place_of<PASS>(a);
  const int tokens = max(p.t_end - p.t_lo, 0), chunks = (tokens + kChunk - 1) / kChunk;
  const long long bh = (long long)p.b * io.H + p.h, nbh = (long long)io.B * io.H, sn = (long long)io.dk * io.dv;
  if (PASS == kJoin) wait_previous();

  auto wait = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity & 1u, stop); };
  auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(i, parity)); };
  auto arrive = [&](int i) {  // once for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };

  if (warp == 0) {
    // ---- decays, then copies ----
    const float* g = io.g ? io.g + p.b * io.g_bs + p.h : nullptr;
    float next[4];
    auto ask = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = c * kChunk + lane * 4 + i;
        next[i] = g && t < tokens ? g[(p.t_lo + t) * io.g_ts] : 0.f;
      }
    };
    ask(0);
    double total = 0.0;
    int load = 0;
    for (int c = 0; c < chunks; ++c) {
      if (!wait_all(kDecayEmpty + (c & 1), uint32_t(c >> 1) + 1)) break;
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = next[i];
      if (c + 1 < chunks) ask(c + 1);
      Decays& d = decays[c & 1];
      double up[4], down[4];  // sums up to and after each token of the lane's
      up[0] = e[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) up[i] = up[i - 1] + double(e[i]);
      down[3] = 0.0;
#pragma unroll
      for (int i = 2; i >= 0; --i) down[i] = down[i + 1] + double(e[i + 1]);
      double before = up[3], after = up[3];  // scans of the lanes' sums
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const double x = __shfl_up_sync(0xFFFFFFFFu, before, m), y = __shfl_down_sync(0xFFFFFFFFu, after, m);
        if (lane >= m) before += x;
        if (lane + m < 32) after += y;
      }
      const double all = __shfl_sync(0xFFFFFFFFu, before, 31);
      double left = __shfl_up_sync(0xFFFFFFFFu, before, 1), right = __shfl_down_sync(0xFFFFFFFFu, after, 1);
      if (lane == 0) left = 0.0;
      if (lane == 31) right = 0.0;
      const double log2e = 1.4426950408889634;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = lane * 4 + i;
        d.each[t] = exp2f(float(double(e[i]) * log2e));
        d.from[t] = finite_exp2(float((left + up[i]) * log2e));
        d.to[t] = c * kChunk + t < tokens ? finite_exp2(float((right + down[i]) * log2e)) : 0.f;
      }
      if (lane == 0) d.all = finite_exp2(float(all * log2e));
      total += all;
      arrive(kDecayFull + (c & 1));
      bool ok = true;
      if (lane == 0) {
        for (int i = 3 - kLoads; i < 3 && ok; ++i, ++load) {
          const int slot = load % kSlots;
          ok = wait(kEmpty + slot, uint32_t(load / kSlots) + 1);
          if (!ok) break;
          const uint32_t dst = base + uint32_t(slot) * kSlot;
          const int boxes = i == 2 ? kBoxesV : kBoxesK, t = p.t_lo + c * kChunk;
          mbar_expect_tx(bar(kFull + slot), uint32_t(boxes * kBox));
          for (int x = 0; x < boxes; ++x)
            tma_load_4d(dst + uint32_t(x * kBox), i == 0 ? &tm.q : i == 1 ? &tm.k : &tm.v, x * 64, i == 2 ? p.h : p.hk, t,
                        p.b, bar(kFull + slot));
          issued[slot] = issued[slot] + 1u;
        }
      }
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
    }
    if (PASS == kReduce && lane == 0) a.ws_g[p.seg * nbh + bh] = float(total);
  } else if (warp == 1) {
    // ---- MMAs ----
    if (lane == 0) {
      int slices = 0;  // so far
      bool ok = true;
      for (int c = 0; c < chunks && ok; ++c) {
        const int n = min(kChunk, tokens - c * kChunk), first = c * kLoads;
        const int iq = first, ik = first + kLoads - 2, iv = first + kLoads - 1;  // loads
        const uint32_t sq = base + uint32_t(iq % kSlots) * kSlot, sk = base + uint32_t(ik % kSlots) * kSlot,
                       sv = base + uint32_t(iv % kSlots) * kSlot;
        if (n < kChunk && !(ok = wait(kCut, 0))) break;
        if (!(ok = wait(kFull + ik % kSlots, uint32_t(ik / kSlots)))) break;
        if (PASS != kReduce) {
          if (!(ok = wait(kFull + iq % kSlots, uint32_t(iq / kSlots)))) break;
          if (!(ok = wait(kScoreEmpty, uint32_t(c) + 1))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t off = uint32_t(kk / 4 * kBox + kk % 4 * 32);
            mma1(tmem + kScore, sw128_desc(sq + off), sw128_desc(sk + off), kk > 0, tile_idesc(128, false, false));
          }
          mma_commit(bar(kScoreFull));
          if (!(ok = wait(kStateFull, uint32_t(c)))) break;
          if (!(ok = wait(kOutEmpty, uint32_t(c) + 1))) break;
          tc_fence_after();
          const uint32_t ss = base + L::off_state;
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma1(tmem + kOutState, sw128_desc(sq + uint32_t(kk / 4 * kBox + kk % 4 * 32)),
                 mn_box_desc(ss + uint32_t(kk * 2048), DK * 128), kk > 0, tile_idesc(DV, false, true));
          mma_commit(bar(kStateEmpty));
          mma_commit(bar(kEmpty + iq % kSlots));
        }
        if (!(ok = wait(kSumEmpty, uint32_t(c) + 1))) break;
        const int ns = (n + kSlice - 1) / kSlice;
        for (int s = 0; s < ns; ++s, ++slices) {
          const int b = slices & 1;
          if (!(ok = wait(kPartFull + b, uint32_t(slices >> 1)))) break;
          tc_fence_after();
          const uint32_t sp = base + L::off_parts + uint32_t(b * 3 * L::part);
#pragma unroll
          for (int i = 0; i < 3; ++i)
            mma1(tmem + kSum, mn_box_desc(sk + uint32_t(s * 2048), kBox), mn_box_desc(sp + uint32_t(i * L::part), kSlice * 128),
                 s > 0 || i > 0, tile_idesc(DV, true, true));
          mma_commit(bar(kPartEmpty + b));
        }
        if (!ok) break;
        mma_commit(bar(kSumFull));
        mma_commit(bar(kEmpty + ik % kSlots));
        if (PASS != kReduce) {
          if (!(ok = wait(kMaskFull, uint32_t(c)))) break;
          if (!(ok = wait(kFull + iv % kSlots, uint32_t(iv / kSlots)))) break;
          tc_fence_after();
          const uint32_t sm = base + L::off_mask;
#pragma unroll
          for (int kk = 0; kk < kChunk / 16; ++kk)
            mma1(tmem + kOutChunk, sw128_desc(sm + uint32_t(kk / 4 * kBox + kk % 4 * 32)),
                 mn_box_desc(sv + uint32_t(kk * 2048), kBox), kk > 0, tile_idesc(DV, false, true));
          mma_commit(bar(kMaskEmpty));
          mma_commit(bar(kOutFull));
        }
        mma_commit(bar(kEmpty + iv % kSlots));
      }
      mma_commit(bar(kDrain));
      mbar_wait_teardown(bar(kDrain), 0);
    }
  } else if (warp < kStateWarp) {
    // ---- masked products, then o ----
    if (PASS != kReduce) {
      const int quad = warp & 3, half = (warp - kMaskWarp) >> 2;
      const int row = quad * 32 + lane;
      const uint32_t lanes = uint32_t(quad * 32) << 16;
      // Blocks of 32 columns up to the diagonal's: the first half of the warps takes the later ones.
      const int cut = (quad + 1) / 2, b_hi = half ? cut - 1 : quad, b_lo = half ? 0 : cut;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(io.o) +
                           (((long long)p.b * io.T + p.t_lo + row) * io.H + p.h) * io.dv + half * (DV / 2);
      for (int c = 0; c < chunks; ++c) {
        const int n = min(kChunk, tokens - c * kChunk);
        if (!wait_all(kDecayFull + (c & 1), uint32_t(c >> 1))) break;
        const Decays& d = decays[c & 1];
        if (!wait_all(kScoreFull, uint32_t(c))) break;
        tc_fence_after();
        if (!wait_all(kMaskEmpty, uint32_t(c) + 1)) break;
        float f = io.scale;  // A_ij scale of the column last passed
        if (half) {          // from the diagonal to this warp's columns
          f = io.scale;
          for (int j = quad * 32 + 31; j > b_hi * 32 + 31; --j) f = j <= row ? f * d.each[j] : f;
        }
        for (int b = b_hi; b >= b_lo; --b) {
          uint32_t r[32];
          tmem_load32(tmem + lanes + kScore + uint32_t(b * 32), r);
          const bool diagonal = b == quad;
          const uint32_t dst = base + L::off_mask + uint32_t(b / 2 * kBox);
#pragma unroll
          for (int w = 3; w >= 0; --w) {
            float v[8];
#pragma unroll
            for (int i = 7; i >= 0; --i) {
              const int j = w * 8 + i;  // column in the block
              // f: A of column j.  Past the columns of the block before, only the entry's own decay is left to apply.
              v[i] = diagonal && j > lane ? 0.f : f * __uint_as_float(r[j]);
              if (!diagonal || j <= lane) f *= d.each[b * 32 + j];
            }
            shared_store(dst + swizzled(row, (b & 1) * 4 + w), Piece<__nv_bfloat16>::pack(v));
          }
        }
        async_proxy_fence();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kScoreEmpty));
          mbar_arrive(bar(kMaskFull));
        }
        const float from = d.from[row] * io.scale;
        if (!wait_all(kOutFull, uint32_t(c))) break;
        tc_fence_after();
        const bool here = p.t_lo + c * kChunk + row < p.t_hi, live = row < n;
#pragma unroll
        for (int x = 0; x < DV / 2; x += 16) {
          uint32_t r1[16], r2[16];
          tmem_load16(tmem + lanes + kOutState + uint32_t(half * (DV / 2) + x), r1);
          tmem_load16(tmem + lanes + kOutChunk + uint32_t(half * (DV / 2) + x), r2);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = live ? fmaf(from, __uint_as_float(r1[8 * k + i]), __uint_as_float(r2[8 * k + i])) : 0.f;
            if (here && half * (DV / 2) + x + 8 * k < io.dv)
              *reinterpret_cast<uint4*>(out + x + 8 * k) = Piece<__nv_bfloat16>::pack(v);
          }
        }
        out += (long long)kChunk * io.H * io.dv;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kOutEmpty));
          mbar_arrive(bar(kDecayEmpty + (c & 1)));
        }
      }
    }
  } else {
    // ---- weighted v, then the state ----
    constexpr int kCols = DV / 2;
    const int quad = warp & 3, half = (warp - kStateWarp) >> 2, tid = threadIdx.x - kStateWarp * 32;
    const int row = quad * 32 + lane, c0 = half * kCols;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const bool rows = row < DK;  // this warp has rows of the state
    float s[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) s[i] = 0.f;
    const float* src = PASS == kJoin ? a.ws_s + (p.seg * nbh + bh) * sn
                       : PASS == kWhole && io.state && p.slot >= 0 ? io.state + ((long long)p.slot * io.H + p.h) * sn
                                                                   : nullptr;
    if (src && row < io.dk) {
      src += (long long)row * io.dv + c0;
      if (a.vec_s) {
#pragma unroll
        for (int i = 0; i < kCols; i += 4)
          if (c0 + i < io.dv) {
            const float4 w = *reinterpret_cast<const float4*>(src + i);
            s[i] = w.x, s[i + 1] = w.y, s[i + 2] = w.z, s[i + 3] = w.w;
          }
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (c0 + i < io.dv) s[i] = src[i];
      }
    }
    auto show_state = [&] {  // as q reads it
      if (rows) {
#pragma unroll
        for (int i = 0; i < kCols; i += 8) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = s[i + k];
          const int col = c0 + i;
          shared_store(base + L::off_state + uint32_t(col / 64 * DK * 128) + swizzled(row, col / 8 % 8),
                       Piece<__nv_bfloat16>::pack(v));
        }
      }
      async_proxy_fence();
      arrive(kStateFull);
    };
    if (PASS != kReduce && chunks > 0) show_state();
    int slices = 0;
    for (int c = 0; c < chunks; ++c) {
      const int n = min(kChunk, tokens - c * kChunk), first = c * kLoads, ik = first + kLoads - 2, iv = first + kLoads - 1;
      const uint32_t sk = base + uint32_t(ik % kSlots) * kSlot, sv = base + uint32_t(iv % kSlots) * kSlot;
      if (!wait_all(kFull + iv % kSlots, uint32_t(iv / kSlots))) break;
      if (n < kChunk) {  // what lies behind the last token may be anything, and 0 times it is not 0
        if (!wait_all(kFull + ik % kSlots, uint32_t(ik / kSlots))) break;
        for (int i = tid; i < (kChunk - n) * 8; i += 256) {
          const uint32_t at = uint32_t((n + i / 8) * 128 + i % 8 * 16);
#pragma unroll
          for (int x = 0; x < kBoxesK; ++x) shared_store(sk + uint32_t(x * kBox) + at, make_uint4(0, 0, 0, 0));
#pragma unroll
          for (int x = 0; x < kBoxesV; ++x) shared_store(sv + uint32_t(x * kBox) + at, make_uint4(0, 0, 0, 0));
        }
        async_proxy_fence();
        arrive(kCut);
        if (!wait_all(kCut, 0)) break;  // the others of this group, whose rows are read below
      }
      if (!wait_all(kDecayFull + (c & 1), uint32_t(c >> 1))) break;
      const Decays& d = decays[c & 1];
      bool ok = true;
      for (int t0 = 0; t0 < n; t0 += kSlice, ++slices) {
        const int b = slices & 1;
        if (!(ok = wait_all(kPartEmpty + b, uint32_t(slices >> 1) + 1))) break;
        constexpr int PR = DV / 8;  // pieces of a token
        if (tid < kSlice * PR) {
          const int t = tid / PR, piece = tid % PR;
          const float w = d.to[t0 + t];
          float x[8];
          Piece<__nv_bfloat16>::load(shared_load(sv + uint32_t(piece / 8 * kBox) + swizzled(t0 + t, piece % 8)), x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= w;
          const uint32_t dst = base + L::off_parts + uint32_t(b * 3 * L::part + piece / 8 * kSlice * 128) + swizzled(t, piece % 8);
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const uint4 h = Piece<__nv_bfloat16>::pack(x);
            shared_store(dst + uint32_t(k * L::part), h);
            if (k == 2) break;
            float y[8];
            Piece<__nv_bfloat16>::load(h, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] -= y[i];
          }
        }
        async_proxy_fence();
        arrive(kPartFull + b);
      }
      if (!ok) break;
      const float all = d.all;
      arrive(kDecayEmpty + (c & 1));
      if (!wait_all(kSumFull, uint32_t(c))) break;
      tc_fence_after();
      if (rows) {
#pragma unroll
        for (int i = 0; i < kCols; i += 16) {
          uint32_t r[16];
          tmem_load16(tmem + lanes + kSum + uint32_t(c0 + i), r);
#pragma unroll
          for (int k = 0; k < 16; ++k) s[i + k] = fmaf(all, s[i + k], __uint_as_float(r[k]));
        }
      }
      tc_fence_before();
      arrive(kSumEmpty);
      if (PASS != kReduce && c + 1 < chunks) {
        if (!wait_all(kStateEmpty, uint32_t(c))) break;
        show_state();
      }
    }
    float* dst = PASS == kReduce                              ? a.ws_s + (p.seg * nbh + bh) * sn
                 : p.last && io.state_out && p.slot >= 0 ? io.state_out + ((long long)p.slot * io.H + p.h) * sn
                                                              : nullptr;
    if (dst && row < io.dk) {
      dst += (long long)row * io.dv + c0;
      if (a.vec_s) {
#pragma unroll
        for (int i = 0; i < kCols; i += 4)
          if (c0 + i < io.dv) *reinterpret_cast<float4*>(dst + i) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (c0 + i < io.dv) dst[i] = s[i];
      }
    }
  }

  // No token here: o is 0.
  if (PASS != kReduce) {
    const int t0 = p.t_lo + chunks * kChunk, pieces = io.dv / 8;
    for (long long i = threadIdx.x; i < (long long)(p.t_hi - t0) * pieces; i += kTileThreads)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(io.o) +
                                (((long long)p.b * io.T + t0 + i / pieces) * io.H + p.h) * io.dv + i % pieces * 8) =
          make_uint4(0, 0, 0, 0);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (threadIdx.x == 0 && *stop) {
    for (int i = 0; i < kSlots; ++i)
      if (issued[i] > 0) mbar_wait_teardown(bar(kFull + i), (issued[i] - 1u) & 1u);
    if (a.dev_err) atomicOr(a.dev_err, SDM_DEV_TIMEOUT);
  }
}

// [B, T, heads, d] with these strides in boxes of 128 tokens x 64 columns of a head; reads are zero outside.
bool head_map(CUtensorMap* map, const void* p, int B, int T, int heads, int d, long long bs, long long ts) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(T), cuuint64_t(B)};
  const cuuint64_t strides[3] = {cuuint64_t(d) * 2, cuuint64_t(ts) * 2, cuuint64_t(B > 1 ? bs : ts) * 2};
  const cuuint32_t box[4] = {64, 1, kChunk, 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, int PASS>
int launch_pass(const TileMaps& tm, const LinearArgs& a, cudaStream_t s) {
  auto fn = tile_kernel<DK, DV, PASS>;
  constexpr int bytes = Tiles<DK, DV>::bytes;
  static PerDevice ready;
  if (ready.get([&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? 1 : -1;
      }) < 0)
    return SDM_ECUDA;
  const long long blocks = (long long)a.io.H * a.io.B * (PASS == kReduce ? a.segments - 1 : a.segments);
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = size_t(bytes);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PASS == kJoin ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, tm, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

template <int DK, int DV>
int launch_sizes(const TileMaps& tm, const LinearArgs& a, cudaStream_t s) {
  if (a.segments <= 1) return launch_pass<DK, DV, kWhole>(tm, a, s);
  int st = launch_pass<DK, DV, kReduce>(tm, a, s);
  if (st == SDM_OK) st = launch_front(a, s);
  return st == SDM_OK ? launch_pass<DK, DV, kJoin>(tm, a, s) : st;
}

}  // namespace

// A CTA of the tile kernel fills an SM and takes a chunk in about the time of 64 to 128 KB of HBM traffic of its share, so
// 152 of them are what the card runs at once.
void cut_tiles(int B, int T, int H, int* segments, int* segment) {
  const long long units = (long long)B * H, chunks = (T + kChunk - 1) / kChunk;
  long long n = units * 2 > 152 ? 1 : 152 / units;
  n = n < chunks / 2 ? n : chunks / 2;
  if (n < 3) n = 1;
  const long long per = (chunks + n - 1) / n;
  *segments = n > 1 ? int((chunks + per - 1) / per) : 1;
  *segment = n > 1 ? int(per * kChunk) : T;
}

int launch_tiles(LinearArgs a, cudaStream_t s) {
  const sdm_linear_args& io = a.io;
  a.vtiles = 1;
  TileMaps tm = {};
  if (!head_map(&tm.q, io.q, io.B, io.T, io.Hk, io.dk, io.q_bs, io.q_ts) ||
      !head_map(&tm.k, io.k, io.B, io.T, io.Hk, io.dk, io.k_bs, io.k_ts) ||
      !head_map(&tm.v, io.v, io.B, io.T, io.H, io.dv, io.v_bs, io.v_ts))
    return SDM_ECUDA;
  if (io.dk <= 64) return io.dv <= 64 ? launch_sizes<64, 64>(tm, a, s) : launch_sizes<64, 128>(tm, a, s);
  return io.dv <= 64 ? launch_sizes<128, 64>(tm, a, s) : launch_sizes<128, 128>(tm, a, s);
}

}  // namespace sdm
