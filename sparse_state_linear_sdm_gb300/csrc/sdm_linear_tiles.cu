// Linear attention over prompts in chunks of 128 tokens on the tcgen05 tensor cores (bf16, dk up to 128, dv up to 256).
//
// With A_ij the product of the decays of tokens j+1 .. i of a chunk, S the state in front of it and G the products from its start:
//
//   o_i = scale (sum_{j<=i} A_ij (q_i k_j) v_j  +  G_i q_i S)
//   S'  = G_last S + sum_j k_j (A_last,j v_j)^T
//
// Four products a chunk: q k^T, q S, (A q k^T) v and (A v)^T k, the last one the state transposed.  A CTA takes a
// sequence's head, its state in registers (fp32, 64 a thread), and walks its chunks.  Warps by role: TMA; the MMAs of
// o; those of the state; decays; eight that turn q k^T into the masked bf16 products, scale q S by G and write o; eight
// that update the state; the two eights share the weighting of v.  k, q and v of two chunks have a slot of 32 KB
// each.  An MMA of 128 x 128 x 16 whose operands both lie in shared memory waits for them (64 bytes a clock: 128
// clocks instead of 64), so the masked products and the weighted v are first operands out of TMEM.
//
// HBM would bound it (128 KB a chunk: 8 prompts of 4096 x 16 heads of 128 in 81 us), the work between the products does:
// 122 to 133 us there, by GPU (the same code), 3.8 us a chunk and SM.  (182 with every operand in shared memory and one
// group for v and the state; 145 with the first slices of v weighed by the state's group in the chunk itself: 36 % of the
// issue slots then, a third of the stalls instruction fetches of five roles' code.)  One prompt of 32,768 x 8 heads, in 19
// segments: 114 to 119 us.
//
// What is rounded to bf16: the masked products and the state as q reads it, as an MMA takes them (each half a unit, as o
// itself).  The state is not: A v is cut into three bf16 parts whose products are summed in fp32 (two parts
// leave 3e-6 of the state, three 1e-8), which costs two more MMAs of six a chunk and no byte.
// The A_ij of a row are formed by one product after the other from the diagonal on, so a decay of 0 leaves 0 before it
// and no difference of sums is taken; G and A_last,j come from sums of g in two floats.
#include "sdm_linear.cuh"
#include "sdm_tcgen05.cuh"

namespace sdm {
namespace {

constexpr int kChunk = 128;
constexpr int kSlot = 32768;             // 128 tokens of 128 columns: two boxes of 64 columns
constexpr int kBox = kChunk * 128;       // bytes of a box
constexpr int kSlots = 6;                // two chunks
constexpr int kSlice = 32;               // tokens of a weighted slice of v: two K steps
// Warps: copies; the MMAs of o; those of the state; decays; and two groups of eight.
constexpr int kTileThreads = 32 * 20;
constexpr int kMaskWarp = 4, kStateWarp = 12;
// Slices of a chunk that the group of o weighs, the first ones, while the tensor cores make o of the chunk before; the
// state's group has the rest.
constexpr int kEarlySlices = 2;
static_assert(kChunk / kSlice == 4 && kEarlySlices == 2, "two buffers, each group's slices in either");

enum Bar {
  kFull = 0, kEmpty = kSlots,     // slots
  kScoreFull = 2 * kSlots,        // q k^T
  kReadFull,                      // q S
  kMaskFull,                      // the masked products, in the place of q k^T
  kOutFull, kOutEmpty,            // o
  kStateFull, kStateEmpty,        // the state as q reads it
  kPartFull, kPartEmpty = kPartFull + 2,  // weighted slices: the buffer's, and those of a chunk one by one
  kSumFull = kPartEmpty + kChunk / kSlice, kSumEmpty,  // k^T (A v)
  kStaged,                        // o has left the slot of q, of even and of odd chunks: the copies may be late by two
  kDone = kStaged + 2,            // the MMAs of o, of even and of odd chunks
  kDecayFull = kDone + 2, kDecayEmpty = kDecayFull + 2,  // of even and of odd chunks
  kEachEmpty = kDecayEmpty + 2,
  kCut,                // tokens past the end cleared
  kDrain, kBars = kDrain + 2
};

struct Decays {
  float each[kChunk];  // e^g of a chunk
  struct Chunk {
    float block[kChunk];       // products from the start of each token's block of 32 up to it
    float rest[kChunk];        // and those after it up to the block's end; 0 past the sequence's
    float before[4], after[4]; // products of the blocks before and after each
    float all, pad[3];
  } of[2];  // even chunks, odd ones
};

template <int DK, int DV>
struct Tiles {
  static constexpr int off_state = kSlots * kSlot;
  static constexpr int off_decays = off_state + DK * DV * 2;
  static constexpr int off_bars = off_decays + int(sizeof(Decays));
  static constexpr int bytes = off_bars + (kBars * 8 + 32 + 15) / 16 * 16;
  static_assert(bytes <= 227 * 1024, "shared memory of a block");
};

// TMEM columns.  Of each 32 of q k^T the masked products take 16; a slice's three parts are 16 columns each.
constexpr uint32_t kScore = 0, kOut = 128, kSum = 256, kParts = 384, kPartCols = kSlice / 2;

struct TileMaps {
  CUtensorMap q, k, v, o;
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
// The whole warp calls these; one lane of it, always the same, issues the MMA or the commit.
__device__ __forceinline__ void mma1(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xFFFFFFFF;\n setp.ne.b32 p, %3, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %4, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(accumulate), "r"(id)
      : "memory");
}
// A from TMEM: 16 bf16 of a row in eight columns.
__device__ __forceinline__ void mma1_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xFFFFFFFF;\n setp.ne.b32 p, %3, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(accumulate), "r"(id)
      : "memory");
}
__device__ __forceinline__ void commit1(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// 16 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store4(uint32_t taddr, const uint4& a) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w)
               : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return uint32_t(row * 128 + ((piece ^ (row & 7)) << 4)); }
__device__ __forceinline__ void shared_store(uint32_t p, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, int x, int y, int z, int w, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
               : "memory");
}
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A sum in two floats: as good as one in 64 bits here, and the card adds few of those.
struct Sum {
  float hi, lo;
  __device__ __forceinline__ Sum operator+(const Sum& o) const {
    const float s = hi + o.hi, z = s - hi;
    return {s, (lo + o.lo) + ((hi - (s - z)) + (o.hi - z))};
  }
  __device__ __forceinline__ Sum from_lane(int lane) const {
    return {__shfl_sync(0xFFFFFFFFu, hi, lane & 31), __shfl_sync(0xFFFFFFFFu, lo, lane & 31)};
  }
  __device__ __forceinline__ float exp() const { return at_most_finite(exp2f(fmaf(hi, kLog2e, lo * kLog2e))); }
};

// One copy of the loop: the roles' code competes for the instruction cache.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* stop, unsigned long long limit_ns) {
  return mbar_wait(bar, parity, stop, limit_ns);
}

// ---- values of v that are not finite ----
//
// 0 times one is not 0, so the masked products carry it to the tokens of its chunk that come before it.  Its column of the
// state is NaN from then on, which shows at the end, and those tokens' outputs are then formed again, token by token from the
// state that the sequence (the segment) begins with: 870 us instead of 125 where each of 8 prompts of 4096 x 16 heads of 128
// has such a token.  Calls without one take what they took without this (121 us then and 123 now on one GPU; 129 to 137
// where a warp looks every chunk over).

// The state in front of the first token.
template <int PASS>
__device__ __forceinline__ const float* front_state(const LinearArgs& a, const Place& p) {
  const sdm_linear_args& io = a.io;
  const long long sn = (long long)io.dk * io.dv;
  if (PASS == kJoin) return a.ws_s + (((long long)p.seg * io.B + p.b) * io.H + p.h) * sn;
  return PASS == kWhole && io.state && p.slot >= 0 ? io.state + ((long long)p.slot * io.H + p.h) * sn : nullptr;
}
// A warp's four columns, the c0-th on (with eight, whose registers spill, the kernel's other code came out slower too: 128 us).
// A lane has rows lane, lane + 32 ...
template <int DK, int PASS>
__device__ void form_columns(const LinearArgs& a, const Place& p, int c0) {
  constexpr int N = DK / 32, kAhead = 4;  // tokens asked for at a time
  const sdm_linear_args& io = a.io;
  const float* src = front_state<PASS>(a, p);
  const int lane = threadIdx.x & 31, tokens = p.t_end - p.t_lo, dk8 = (io.dk + 7) / 8 * 8;
  typedef const __nv_bfloat16* In;
  const In q = In(io.q) + p.b * io.q_bs + p.t_lo * io.q_ts + (long long)p.hk * dk8;
  const In k = In(io.k) + p.b * io.k_bs + p.t_lo * io.k_ts + (long long)p.hk * dk8;
  const In v = In(io.v) + p.b * io.v_bs + p.t_lo * io.v_ts + (long long)p.h * a.o_dv + c0;
  const float* g = io.g ? io.g + p.b * io.g_bs + p.t_lo * io.g_ts + p.h : nullptr;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(io.o) + (((long long)p.b * io.T + p.t_lo) * io.H + p.h) * a.o_dv + c0;
  const long long os = (long long)io.H * a.o_dv;

  int first[4];  // of each column, or the tokens' number
#pragma unroll
  for (int j = 0; j < 4; ++j) first[j] = tokens;
  for (int t0 = 0; t0 < tokens; t0 += 32) {
    uint2 w = make_uint2(0, 0);
    if (t0 + lane < tokens) w = *reinterpret_cast<const uint2*>(v + (t0 + lane) * io.v_ts);
    const uint32_t r[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, (r[j / 2] >> (j % 2 * 16) & 0x7F80u) == 0x7F80u);
      if (hit && first[j] == tokens) first[j] = t0 + __ffs(hit) - 1;
    }
  }
  int from = tokens, to = 0;  // tokens whose outputs are formed again
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (first[j] == tokens) first[j] = 0;
    if (first[j] % kChunk) from = min(from, first[j] / kChunk * kChunk), to = max(to, first[j]);
  }

  float s[N][4];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = lane + 32 * i;
      s[i][j] = src && r < io.dk && c0 + j < io.dv ? src[(long long)r * io.dv + c0 + j] : 0.f;
    }
  for (int t0 = 0; t0 < to; t0 += kAhead) {
    __nv_bfloat16 kr[kAhead][N];
    uint2 vr[kAhead];
    float gr[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int t = min(t0 + x, tokens - 1);
      vr[x] = *reinterpret_cast<const uint2*>(v + t * io.v_ts);
      gr[x] = g ? g[t * io.g_ts] : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) kr[x][i] = lane + 32 * i < io.dk ? k[t * io.k_ts + lane + 32 * i] : __nv_bfloat16(0.f);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int t = t0 + x;
      if (t >= to) break;
      const float e = at_most_finite(expf(gr[x]));
      const float f[4] = {__uint_as_float(vr[x].x << 16), __uint_as_float(vr[x].x & 0xFFFF0000u), __uint_as_float(vr[x].y << 16),
                          __uint_as_float(vr[x].y & 0xFFFF0000u)};
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(e, s[i][j], to_f32(kr[x][i]) * f[j]);
      if (t < from) continue;
      float qr[N];
#pragma unroll
      for (int i = 0; i < N; ++i) qr[i] = lane + 32 * i < io.dk ? to_f32(q[t * io.q_ts + lane + 32 * i]) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) y = fmaf(qr[i], s[i][j], y);
#pragma unroll
        for (int m = 16; m > 0; m /= 2) y += __shfl_xor_sync(0xFFFFFFFFu, y, m);
        if (lane == j && t >= first[j] / kChunk * kChunk && t < first[j]) from_f32(y * io.scale, o + t * os + j);
      }
    }
  }
}

template <int DK, int PASS>
__device__ __noinline__ void form_again(const LinearArgs& a) {
  const Place p = place_of<PASS>(a);
  const int c0 = p.vt * kTileColumns, warp = threadIdx.x >> 5;
  for (int c = warp * 4; c < min(kTileColumns, a.o_dv - c0); c += kStateWarp * 4) form_columns<DK, PASS>(a, p, c0 + c);
}

// Every wait is bounded; one that runs out stops the CTA, which waits for the copies and MMAs in flight, frees TMEM and
// reports SDM_DEV_TIMEOUT.  A new state is written whole or not at all.
template <int DK, int DV, int PASS>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ TileMaps tm, const __grid_constant__ LinearArgs a) {
  typedef Tiles<DK, DV> L;
  constexpr int kBoxesK = DK / 64, kBoxesV = DV / 64;
  constexpr int kLoads = PASS == kReduce ? 2 : 3;  // slots a chunk takes
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's atoms; there is no room to align it here
  const uint32_t base = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::off_bars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  volatile int* stop = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* issued = tmem_slot + 2;
  Decays& d = *reinterpret_cast<Decays*>(smem + L::off_decays);
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const sdm_linear_args& io = a.io;

  if (PASS == kReduce) allow_next();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      int n = 1;
      if (i == kMaskFull || i == kStaged || i == kStaged + 1 || i == kOutEmpty || i == kStateFull || i == kPartFull || i == kPartFull + 1 ||
          i == kSumEmpty || i == kCut)
        n = 8;  // the warps of a group
      if (i == kEachEmpty) n = 8;
      if (i == kDecayEmpty || i == kDecayEmpty + 1) n = 16;
      mbar_init(bar(i), uint32_t(n));
    }
    *stop = (base & 1023u) != 0;
    for (int i = 0; i < kSlots; ++i) issued[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Place p = place_of<PASS>(a);
  const int tokens = max(p.t_end - p.t_lo, 0), chunks = (tokens + kChunk - 1) / kChunk;
  const int v0 = p.vt * kTileColumns, dv = min(kTileColumns, io.dv - v0);  // this CTA's columns of v
  const long long bh = (long long)p.b * io.H + p.h, nbh = (long long)io.B * io.H, sn = (long long)io.dk * io.dv;
  if (PASS == kJoin) wait_previous();

  auto wait = [&](int i, uint32_t parity) {
    return mbar_test(bar(i), parity & 1u) || wait_on(bar(i), parity & 1u, stop, a.stall.wait_ns);
  };
  auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(i, parity)); };
  auto arrive = [&](int i) {  // once for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };

  // Load i of chunk c: its slot, the turn of it, its address.
  auto slot = [&](int c, int i) { return (c & 1) * 3 + i; };
  auto turn = [&](int c) { return uint32_t(c >> 1); };
  auto place = [&](int slot) { return base + uint32_t(slot) * kSlot; };

  // Either group of eight: slice s of chunk c weighted and cut into its three parts, a column of v a thread.
  const int quad = warp & 3, half = (warp - kMaskWarp) >> 2 & 1;
  const int col = quad * 32 + lane;
  const uint32_t lanes = uint32_t(quad * 32) << 16;
  auto weigh = [&](int c, int s, uint32_t sv) {
    // Before it the buffer had slice s - 2, or s + 2 of the chunk before.  A wait sees one phase ahead and one behind, and either
    // group may be a whole chunk away from the other's slices, so each slice has a barrier of its own.
    const int b = s & 1;
    if (!(s < 2 ? wait_all(kPartEmpty + s + 2, uint32_t(c) + 1) : wait_all(kPartEmpty + s - 2, uint32_t(c)))) return false;
    tc_fence_after();
    if (quad * 32 < DV) {  // half of the slice's tokens, eight at a time
      const Decays::Chunk& dc = d.of[c & 1];
      const uint64_t after = pack2(dc.after[s], dc.after[s]);  // a slice is a block
#pragma unroll 1
      for (int j = 0; j < kSlice / 2; j += 8) {
        const int t1 = s * kSlice + half * (kSlice / 2) + j;
        const uint32_t at = sv + uint32_t(col / 64 * kBox + t1 * 128 + col % 8 * 2);
        uint64_t x[4];  // tokens in pairs
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t h[2];
#pragma unroll
          for (int k = 0; k < 2; ++k)
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h[k]) : "r"(at + swizzled(2 * i + k, col / 8 % 8)) : "memory");
          const float2 w = *reinterpret_cast<const float2*>(&dc.rest[t1 + 2 * i]);
          x[i] = mul2(pack2(__uint_as_float(uint32_t(h[0]) << 16), __uint_as_float(uint32_t(h[1]) << 16)),
                      mul2(pack2(w.x, w.y), after));
        }
        // The first two parts are the upper halves of what is left, so what they leave is exact.
        const uint64_t minus = pack2(-1.f, -1.f);
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float lo, hi;
            unpack2(x[i], lo, hi);
            const uint32_t l = __float_as_uint(lo), u = __float_as_uint(hi);
            if (k == 2) {
              h[i] = pack_bf16(l, u);
            } else {
              h[i] = __byte_perm(l, u, 0x7632);
              x[i] = fma2(pack2(__uint_as_float(l & 0xFFFF0000u), __uint_as_float(u & 0xFFFF0000u)), minus, x[i]);
            }
          }
          tmem_store4(tmem + lanes + kParts + uint32_t(b * 3 + k) * kPartCols + uint32_t(half * 8 + j / 2),
                      make_uint4(h[0], h[1], h[2], h[3]));
        }
      }
      tmem_stored();
    }
    tc_fence_before();
    arrive(kPartFull + b);
    return true;
  };

  if (warp == 0) {
    // ---- copies: k, q, v of each chunk ----
    if (lane == 0) {
      bool ok = true;
      for (int c = 0; c < chunks && ok; ++c) {
        const int t = p.t_lo + c * kChunk;
        for (int j = 0; j < kLoads; ++j) {  // v, which is weighed early, then k, then q, whose place is free last
          const int i = j == 0 ? kLoads - 1 : j - 1, at = slot(c, i);
          if (a.stall.pass == PASS && int(blockIdx.x) == a.stall.block && c == a.stall.chunk && i == a.stall.load) ok = false;
          // The slot's last load: q's is free when o has left its place, the others' when their MMAs are done.
          if (ok && c > 1) ok = PASS != kReduce && i == 1 ? wait(kStaged + (c & 1), turn(c) + 1) : wait(kEmpty + at, turn(c) + 1);
          if (!ok) break;
          const uint32_t dst = place(at), full = bar(kFull + at);
          const bool value = i == kLoads - 1;
          const CUtensorMap* map = value ? &tm.v : i == 0 ? &tm.k : &tm.q;
          const int boxes = value ? kBoxesV : kBoxesK, head = value ? p.h : p.hk, x = value ? v0 : 0;
          mbar_expect_tx(full, uint32_t(boxes * kBox));
          tma_load_4d(dst, map, x, head, t, p.b, full);
          if (boxes > 1) tma_load_4d(dst + kBox, map, x + 64, head, t, p.b, full);
          issued[at] = issued[at] + 1u;
        }
      }
    }
  } else if (warp == 3) {
    // ---- decays, four tokens a lane ----
    const float* g = io.g ? io.g + p.b * io.g_bs + p.h : nullptr;
    float next[4];
    auto ask = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = c * kChunk + lane * 4 + i;
        const float x = g && t < tokens ? g[(p.t_lo + t) * io.g_ts] : 0.f;
        next[i] = x < -1e30f ? -1e30f : x > 1e30f ? 1e30f : x;  // sums stay finite
      }
    };
    ask(0);
    const Sum zero = {0.f, 0.f};
    Sum total = zero;
    for (int c = 0; c < chunks; ++c) {
      Sum up[4], down[4];  // sums up to and after each token of the lane's
      up[0] = {next[0], 0.f};
      down[3] = zero;
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        up[i] = up[i - 1] + Sum{next[i], 0.f};
        down[3 - i] = down[4 - i] + Sum{next[4 - i], 0.f};
      }
      float each[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) each[i] = at_most_finite(exp2_fast(kLog2e * next[i]));
      if (c + 1 < chunks) ask(c + 1);
      // Scans over eight lanes, a block of 32 tokens, then over the blocks.
      Sum before = up[3], after = up[3];
#pragma unroll
      for (int m = 1; m < 8; m *= 2) {
        const Sum x = before.from_lane(lane - m), y = after.from_lane(lane + m);
        if (lane % 8 >= m) before = before + x;
        if (lane % 8 + m < 8) after = after + y;
      }
      const Sum in_block = before.from_lane(lane | 7);
      Sum earlier = zero, later = zero, all = zero;  // whole blocks
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const Sum x = in_block.from_lane(b * 8);
        if (b < lane / 8) earlier = earlier + x;
        if (b > lane / 8) later = later + x;
        all = all + x;
      }
      Sum left = before.from_lane(lane - 1), right = after.from_lane(lane + 1);
      if (lane % 8 == 0) left = zero;
      if (lane % 8 == 7) right = zero;
      float block[4], rest[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Sum x = left + up[i], y = right + down[i];
        block[i] = x.exp();
        rest[i] = c * kChunk + lane * 4 + i < tokens ? y.exp() : 0.f;
      }
      const float last = all.exp(), start = earlier.exp(), end = later.exp();
      // All of it is computed here and not behind the wait, after which the other warps wait for it.
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("" ::"f"(each[i]), "f"(block[i]), "f"(rest[i]), "f"(start), "f"(end), "f"(last));
      if (!wait_all(kDecayEmpty + (c & 1), turn(c) + 1)) break;
      if (PASS != kReduce && !wait_all(kEachEmpty, uint32_t(c) + 1)) break;
      Decays::Chunk& dc = d.of[c & 1];
      auto put = [&](float* at, const float (&v)[4]) { reinterpret_cast<float4*>(at)[lane] = make_float4(v[0], v[1], v[2], v[3]); };
      put(d.each, each), put(dc.block, block), put(dc.rest, rest);
      if (lane % 8 == 0) dc.before[lane / 8] = start, dc.after[lane / 8] = end;
      if (lane == 0) dc.all = last;
      total = total + all;
      arrive(kDecayFull + (c & 1));
    }
    if (PASS == kReduce && lane == 0 && p.vt == 0) a.ws_g[p.seg * nbh + bh] = total.hi + total.lo;
  } else if (warp == 1) {
    // ---- MMAs of o ----
    if (PASS != kReduce) {
      auto step = [](int kk) { return uint64_t(kk / 4 * kBox + kk % 4 * 32) >> 4; };  // K steps along a row of boxes
      for (int c = 0; c < chunks; ++c) {
        const int ik = slot(c, 0), iq = slot(c, 1), iv = slot(c, 2);
        const uint64_t q = sw128_desc(place(iq)), k = sw128_desc(place(ik)), v_rows = mn_box_desc(place(iv), kBox);
        if (tokens - c * kChunk < kChunk && !wait_all(kCut, 0)) break;
        if (!wait_all(kFull + ik, turn(c)) || !wait_all(kFull + iq, turn(c))) break;
        if (c > 0 && !wait_all(kOutFull, uint32_t(c) - 1)) break;  // the masked products before have been read
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
          mma1(tmem + kScore, q + step(kk), k + step(kk), kk > 0, tile_idesc(128, false, false));
        commit1(bar(kScoreFull));
        if (!wait_all(kStateFull, uint32_t(c)) || !wait_all(kOutEmpty, uint32_t(c) + 1)) break;
        tc_fence_after();
        const uint64_t state = sw128_desc(base + L::off_state);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
          mma1(tmem + kOut, q + step(kk), state + uint64_t((kk / 4 * DV * 128 + kk % 4 * 32) >> 4), kk > 0,
               tile_idesc(DV, false, false));
        commit1(bar(kReadFull));
        commit1(bar(kStateEmpty));
        if (!wait_all(kMaskFull, uint32_t(c)) || !wait_all(kFull + iv, turn(c))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kChunk / 16; ++kk)
          mma1_tmem(tmem + kOut, tmem + kScore + uint32_t(kk / 2 * 32 + kk % 2 * 8), v_rows + uint64_t(kk * 2048 >> 4), 1,
                    tile_idesc(DV, false, true));
        commit1(bar(kOutFull));
        commit1(bar(kDone + (c & 1)));
      }
    }
  } else if (warp == 2) {
    // ---- MMAs of the state ----
    int slices = 0;  // so far
    bool ok = true;
    for (int c = 0; c < chunks && ok; ++c) {
      const int n = min(kChunk, tokens - c * kChunk), ik = slot(c, 0), iv = slot(c, kLoads - 1);
      const uint64_t k_rows = mn_box_desc(place(ik), kBox);
      if (n < kChunk && !wait_all(kCut, 0)) break;
      if (!wait_all(kFull + ik, turn(c)) || !wait_all(kSumEmpty, uint32_t(c) + 1)) break;
      for (int t0 = 0; t0 < n; t0 += kSlice, ++slices) {
        const int b = slices & 1;
        if (!(ok = wait_all(kPartFull + b, uint32_t(slices >> 1)))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kSlice / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 3; ++i)
            mma1_tmem(tmem + kSum, tmem + kParts + uint32_t(b * 3 + i) * kPartCols + uint32_t(kk * 8),
                      k_rows + uint64_t((t0 + kk * 16) * 128 >> 4), t0 > 0 || kk > 0 || i > 0, tile_idesc(DK, false, true));
        commit1(bar(kPartEmpty + t0 / kSlice));
      }
      if (!ok) break;
      commit1(bar(kSumFull));
      // Both groups of MMAs read k, and v is read for both.
      if (PASS != kReduce && !wait_all(kDone + (c & 1), uint32_t(c >> 1))) break;
      commit1(bar(kEmpty + ik));
      commit1(bar(kEmpty + iv));
    }
  } else if (warp < kStateWarp) {
    // ---- masked products, some of weighted v, then o ----
    auto weigh_first = [&](int c) {
      const int n = min(kChunk, tokens - c * kChunk), iv = slot(c, kLoads - 1);
      bool ok = wait_all(kDecayFull + (c & 1), turn(c)) && wait_all(kFull + iv, turn(c)) && (n == kChunk || wait_all(kCut, 0));
#pragma unroll 1
      for (int i = 0; i < kEarlySlices && i * kSlice < n && ok; ++i) ok = weigh(c, i, place(iv));
      return ok;
    };
    if (PASS == kReduce) {
      for (int c = 0; c < chunks; ++c) {
        if (!weigh_first(c)) break;
        arrive(kDecayEmpty + (c & 1));
      }
    } else {
      const int row = col;
      const uint32_t out_at = tmem + lanes + kOut + uint32_t(half * (DV / 2));
      // Blocks of 32 columns up to the diagonal's: the first half of the warps takes the later ones.
      const int cut = (quad + 1) / 2, b_hi = half ? cut - 1 : quad, b_lo = half ? 0 : cut;
      // This warp's part of o lies where q was: 32 rows of DV / 2 columns, 128 or 64 bytes, in their swizzle.
      constexpr int kRowBytes = DV;
      auto staged = [&](int piece) {
        return DV == 128 ? swizzled(lane, piece) : uint32_t(lane * 64 + ((piece ^ (lane >> 1 & 3)) << 4));
      };
      for (int c = -1; c < chunks; ++c) {  // the first round only weighs
        const int n = min(kChunk, tokens - c * kChunk);
        if (c >= 0) {
          const Decays::Chunk& dc = d.of[c & 1];
          if (!wait_all(kScoreFull, uint32_t(c))) break;
          tc_fence_after();
          float f = io.scale * dc.block[row];  // scale A of this row and the last column of the block that is next
          for (int b = quad - 1; b > b_hi; --b) f *= dc.block[b * 32 + 31];
#pragma unroll 1
          for (int b = b_hi; b >= b_lo; --b) {
            uint32_t r[32], pairs[16];
            tmem_load32(tmem + lanes + kScore + uint32_t(b * 32), r);
            if (b == quad) {  // the diagonal's: from there on a product after the other
              const float* each = d.each + b * 32;
              float e = io.scale;
#pragma unroll
              for (int j = 30; j >= 0; j -= 2) {  // columns j, j + 1 of the block
                const float2 w = *reinterpret_cast<const float2*>(each + j);
                const float hi = j + 1 > lane ? 0.f : e * __uint_as_float(r[j + 1]);
                e = j + 1 > lane ? e : e * w.y;
                const float lo = j > lane ? 0.f : e * __uint_as_float(r[j]);
                e = j > lane ? e : e * w.x;
                pairs[j / 2] = pack_bf16(__float_as_uint(lo), __float_as_uint(hi));
              }
            } else {
              const uint64_t both = pack2(f, f);
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 w = *reinterpret_cast<const float4*>(dc.rest + b * 32 + j);
                float x0, x1;
                unpack2(mul2(mul2(pack2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])), pack2(w.x, w.y)), both), x0, x1);
                pairs[j / 2] = pack_bf16(__float_as_uint(x0), __float_as_uint(x1));
                unpack2(mul2(mul2(pack2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])), pack2(w.z, w.w)), both), x0, x1);
                pairs[j / 2 + 1] = pack_bf16(__float_as_uint(x0), __float_as_uint(x1));
              }
              f *= dc.block[b * 32 + 31];
            }
            tmem_store16(tmem + lanes + kScore + uint32_t(b * 32), pairs);
          }
          arrive(kEachEmpty);
          if (!half) {  // nothing above the diagonal
            const uint32_t zeros[16] = {};
            for (int b = quad + 1; b < 4; ++b) tmem_store16(tmem + lanes + kScore + uint32_t(b * 32), zeros);
          }
          // o of the chunk before has long left for memory
          if (c > 0 && lane == 0) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            mbar_arrive(bar(kStaged + ((c - 1) & 1)));
          }
          __syncwarp();
          // q S, on which the chunk's own products are added, takes the decays from the chunk's start.
          const float from = dc.before[quad] * dc.block[row] * io.scale;
          if (!wait_all(kReadFull, uint32_t(c))) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < DV / 2; x += 16) {
            uint32_t r[16];
            tmem_load16(out_at + uint32_t(x), r);
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(from * __uint_as_float(r[i]));
            tmem_store16(out_at + uint32_t(x), r);
          }
          tmem_stored();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(kMaskFull));
            mbar_arrive(bar(kDecayEmpty + (c & 1)));
          }
        }
        if (c + 1 < chunks && !weigh_first(c + 1)) break;
        if (c < 0) continue;
        if (!wait_all(kOutFull, uint32_t(c))) break;
        tc_fence_after();
        const uint32_t patch = place(slot(c, 1)) + uint32_t((half * 4 + quad) * 32 * kRowBytes);
#pragma unroll 1
        for (int x = 0; x < DV / 2; x += 16) {
          uint32_t r[16];
          tmem_load16(out_at + uint32_t(x), r);
          if (n < kChunk && row >= n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = 0;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t* v = r + 8 * k;
            shared_store(patch + staged(x / 8 + k), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                               pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
          }
        }
        tc_fence_before();
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kOutEmpty));
          tma_store_4d(&tm.o, v0 + half * (DV / 2), p.h, p.t_lo + c * kChunk + quad * 32, p.b, patch);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();
      }
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else {
    // ---- weighted v, then the state ----
    // The state lies transposed: a thread has a column of v and half of the rows, s[i] that of row c0 + i.
    constexpr int kCols = DK / 2;
    const int tid = threadIdx.x - kStateWarp * 32, c0 = half * kCols;
    const bool cols = quad * 32 < DV;  // this warp has columns of v
    float s[kCols];  // the state
#pragma unroll
    for (int i = 0; i < kCols; ++i) s[i] = 0.f;
    const float* src = front_state<PASS>(a, p);
    if (src && col < dv) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (c0 + i < io.dk) s[i] = src[(c0 + i) * io.dv + v0 + col];
    }
    bool lost = false;  // the end of a segment before this one
    if (PASS == kJoin && p.last) {
      for (int i = lane; i < p.seg * a.vtiles; i += 32)
        lost |= a.ws_stop[(i / a.vtiles * nbh + bh) * a.vtiles + i % a.vtiles] != 0;
      lost = __any_sync(0xFFFFFFFFu, lost);
    }
    auto show_state = [&] {  // as q reads it
      if (cols) {
#pragma unroll
        for (int i = 0; i < kCols; i += 8) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = s[i + k];
          const int r = c0 + i;
          shared_store(base + L::off_state + uint32_t(r / 64 * DV * 128) + swizzled(col, r / 8 % 8),
                       Piece<__nv_bfloat16>::pack(v));
        }
      }
      async_proxy_fence();
      arrive(kStateFull);
    };
    if (PASS != kReduce && chunks > 0) show_state();
    int c = 0;
    for (; c < chunks; ++c) {
      const int n = min(kChunk, tokens - c * kChunk), ik = slot(c, 0), iv = slot(c, kLoads - 1);
      const uint32_t sk = place(ik), sv = place(iv);
      if (!wait_all(kFull + iv, turn(c))) break;
      if (n < kChunk) {  // what lies behind the last token may be anything, and 0 times it is not 0
        if (!wait_all(kFull + ik, turn(c))) break;
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
      if (!wait_all(kDecayFull + (c & 1), turn(c))) break;
      bool ok = true;
#pragma unroll 1
      for (int i = kEarlySlices; i * kSlice < n && ok; ++i) ok = weigh(c, i, sv);
      if (!ok) break;
      const float all = d.of[c & 1].all;
      arrive(kDecayEmpty + (c & 1));
      if (!wait_all(kSumFull, uint32_t(c))) break;
      tc_fence_after();
      if (cols) {
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
    float zero = 0.f;
#pragma unroll
    for (int i = 0; i < kCols; ++i) zero = fmaf(0.f, s[i], zero);
    if (PASS != kReduce && __syncthreads_or(zero != 0.f)) __syncthreads();  // the new state may lie over the old one
    float* dst = PASS == kReduce                              ? a.ws_s + (p.seg * nbh + bh) * sn
                 : p.last && io.state_out && p.slot >= 0 ? io.state_out + ((long long)p.slot * io.H + p.h) * sn
                                                              : nullptr;
    // After a wait that ran out the state is that of some chunk on the way: the old one stays.
    if (dst && c == chunks && !lost && col < dv) {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (c0 + i < io.dk) dst[(c0 + i) * io.dv + v0 + col] = s[i];
    }
  }

  __syncwarp();
  if (PASS != kReduce && warp < kStateWarp && __syncthreads_or(0)) {  // a state is not finite
    asm volatile("fence.proxy.async;" ::: "memory");  // o has left by copies
    if (!*stop) form_again<DK, PASS>(a);
    __syncthreads();
  }

  // No token here: o is 0.
  if (PASS != kReduce) {
    const int t0 = p.t_lo + chunks * kChunk, pieces = min(kTileColumns, a.o_dv - v0) / 8;
    __nv_bfloat16* row = static_cast<__nv_bfloat16*>(io.o) + ((long long)p.b * io.T * io.H + p.h) * a.o_dv + v0 + lane * 8;
    if (lane < pieces)
      for (int t = t0 + warp; t < p.t_hi; t += kTileThreads / 32)
        *reinterpret_cast<uint4*>(row + (long long)t * io.H * a.o_dv) = make_uint4(0, 0, 0, 0);
  }

  if (warp == 1 || warp == 2) {
    __syncwarp();
    commit1(bar(kDrain + warp - 1));
    mbar_wait_teardown(bar(kDrain + warp - 1), 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  if (PASS == kReduce && threadIdx.x == 0) a.ws_stop[(p.seg * nbh + bh) * a.vtiles + p.vt] = *stop;
  if (threadIdx.x == 0 && *stop) {
    for (int i = 0; i < kSlots; ++i)
      if (issued[i] > 0) mbar_wait_teardown(bar(kFull + i), (issued[i] - 1u) & 1u);
    if (a.dev_err) atomicOr(a.dev_err, SDM_DEV_TIMEOUT);
  }
}

// [B, T, heads, d] with these strides in boxes of some tokens and 64 or 32 columns of a head; reads are zero outside,
// and nothing is written there.
bool head_map(CUtensorMap* map, const void* p, int B, int T, int heads, int d, long long bs, long long ts, int rows = kChunk,
              int cols = 64) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(T), cuuint64_t(B)};
  const cuuint64_t strides[3] = {cuuint64_t(d) * 2, cuuint64_t(ts) * 2, cuuint64_t(B > 1 ? bs : ts) * 2};
  const cuuint32_t box[4] = {cuuint32_t(cols), 1, cuuint32_t(rows), 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
  const long long blocks = (long long)a.vtiles * a.io.H * a.io.B * (PASS == kReduce ? a.segments - 1 : a.segments);
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

// ---- rows off 16 bytes ----
//
// Copied to rows of multiples of eight columns first, and o back: 8 x 2048 x 16 heads with dk 100 and dv 128 take 172 us
// so, and 1,006 token by token.

// q, k and v of the tokens that exist: a block has some tokens of one sequence and one of the three, a warp their heads in
// turn, four of them at a time, a lane two columns.
constexpr int kPadThreads = 256, kPadTokens = 16, kPadRows = 4;
struct PadArgs {
  sdm_linear_args io;
  __nv_bfloat16* to[3];
  int pad[3];  // columns there
};
__global__ void __launch_bounds__(kPadThreads) widen_kernel(const __grid_constant__ PadArgs a) {
  const sdm_linear_args& io = a.io;
  const int which = blockIdx.y, tiles = (io.T + kPadTokens - 1) / kPadTokens;
  const int b = int(blockIdx.x / unsigned(tiles)), t0 = int(blockIdx.x % unsigned(tiles)) * kPadTokens;
  const int n = min(kPadTokens, row_length(io.lengths, b, io.T) - t0);
  const int heads = which == 2 ? io.H : io.Hk, d = which == 2 ? io.dv : io.dk, dp = a.pad[which];
  const long long bs = which == 0 ? io.q_bs : which == 1 ? io.k_bs : io.v_bs, ts = which == 0 ? io.q_ts : which == 1 ? io.k_ts : io.v_ts;
  const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(which == 0 ? io.q : which == 1 ? io.k : io.v) + b * bs + t0 * ts;
  __nv_bfloat16* to = a.to[which] + ((long long)b * io.T + t0) * heads * dp;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = n * heads;
  for (int r0 = warp * kPadRows; r0 < rows; r0 += kPadThreads / 32 * kPadRows)
    for (int c = 2 * lane; c < dp; c += 64) {
      __nv_bfloat162 v[kPadRows];
#pragma unroll
      for (int i = 0; i < kPadRows; ++i) {
        const int r = r0 + i, t = r / heads;
        const __nv_bfloat16* row = from + t * ts + (r - t * heads) * d + c;
        v[i].x = r < rows && c < d ? row[0] : __nv_bfloat16(0.f);
        v[i].y = r < rows && c + 1 < d ? row[1] : __nv_bfloat16(0.f);
      }
#pragma unroll
      for (int i = 0; i < kPadRows; ++i)
        if (r0 + i < rows) *reinterpret_cast<__nv_bfloat162*>(to + (long long)(r0 + i) * dp + c) = v[i];
    }
}
// o out of rows of dp columns.
__global__ void __launch_bounds__(kPadThreads) narrow_kernel(const __nv_bfloat16* from, long long rows, int d, int dp,
                                                             __nv_bfloat16* o) {
  wait_previous();
  const int lane = threadIdx.x & 31;
  const long long r0 = ((long long)blockIdx.x * (kPadThreads / 32) + (threadIdx.x >> 5)) * kPadRows;
  for (int c = 2 * lane; c < d; c += 64) {
    __nv_bfloat162 v[kPadRows];
#pragma unroll
    for (int i = 0; i < kPadRows; ++i)
      if (r0 + i < rows) v[i] = *reinterpret_cast<const __nv_bfloat162*>(from + (r0 + i) * dp + c);
#pragma unroll
    for (int i = 0; i < kPadRows; ++i) {
      if (r0 + i >= rows) break;
      o[(r0 + i) * d + c] = v[i].x;
      if (c + 1 < d) o[(r0 + i) * d + c + 1] = v[i].y;
    }
  }
}

// A CTA of the tile kernel fills an SM, so 152 of them are what the card runs at once.  A chunk takes one about 4 us, and
// 7 over both passes where the sequence is cut, with about 15 us for two more launches and starts.  (50 heads of 4096 tokens in 3
// segments 102 us and 119 whole, of 1024 tokens 44 and 35; 8 heads of 1024 tokens in 4 segments 27 and 35.  Two
// segments gain nothing: 64 heads of 4096 tokens 135 us and 119 whole, in 3 segments 146.  Whole, 51 to 128 heads leave SMs
// idle and take what 51 do.)
void cut_tiles(int B, int T, int H, int dv, int* segments, int* segment) {
  const long long units = (long long)B * H * tile_columns(dv), chunks = ((long long)T + kChunk - 1) / kChunk;
  long long n = 152 / units;
  n = n < chunks / 2 ? n : chunks / 2;
  long long per = n > 1 ? (chunks + n - 1) / n : chunks;
  if (n < 3 || 70 * per + 150 > 41 * chunks) n = 1, per = chunks;
  *segments = n > 1 ? int((chunks + per - 1) / per) : 1;
  *segment = n > 1 ? int(per * kChunk) : T;
}

namespace {
int round8(int d) { return (d + 7) / 8 * 8; }
size_t pad256(size_t n) { return (n + 255) / 256 * 256; }
}  // namespace

size_t padded_bytes(int B, int T, int H, int Hk, int dk, int dv) {
  const size_t tokens = size_t(B) * T * 2;
  return 2 * pad256(tokens * Hk * round8(dk)) + 2 * pad256(tokens * H * round8(dv));
}

int launch_tiles(LinearArgs a, void* pad, cudaStream_t s) {
  const sdm_linear_args given = a.io;
  sdm_linear_args& io = a.io;
  a.vtiles = tile_columns(io.dv);
  if (a.stall.pass < 0) a.stall.wait_ns = kWaitNs;
  a.o_dv = io.dv;
  const int dk = round8(io.dk), dv = round8(io.dv);
  if (pad) {
    if ((long long)io.B * ((io.T + kPadTokens - 1) / kPadTokens) > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
    PadArgs w = {};
    w.io = given;
    uint8_t* at = static_cast<uint8_t*>(pad);
    const size_t tokens = size_t(io.B) * io.T * 2;
    for (int i = 0; i < 3; ++i) {
      w.pad[i] = i == 2 ? dv : dk;
      w.to[i] = reinterpret_cast<__nv_bfloat16*>(at);
      at += pad256(tokens * (i == 2 ? io.H * dv : io.Hk * dk));
    }
    widen_kernel<<<dim3(unsigned(io.B) * unsigned((io.T + kPadTokens - 1) / kPadTokens), 3), kPadThreads, 0, s>>>(w);
    if (last_launch_status() != SDM_OK) return SDM_ECUDA;
    io.q = w.to[0], io.k = w.to[1], io.v = w.to[2], io.o = at;
    io.q_ts = io.k_ts = (long long)io.Hk * dk, io.v_ts = (long long)io.H * dv;
    io.q_bs = io.k_bs = io.q_ts * io.T, io.v_bs = io.v_ts * io.T;
    a.o_dv = dv;
  }
  TileMaps tm = {};
  if (!head_map(&tm.q, io.q, io.B, io.T, io.Hk, dk, io.q_bs, io.q_ts) ||
      !head_map(&tm.k, io.k, io.B, io.T, io.Hk, dk, io.k_bs, io.k_ts) ||
      !head_map(&tm.v, io.v, io.B, io.T, io.H, dv, io.v_bs, io.v_ts) ||
      !head_map(&tm.o, io.o, io.B, io.T, io.H, dv, (long long)io.T * io.H * dv, (long long)io.H * dv, 32,
                io.dv <= 64 ? 32 : 64))
    return SDM_ECUDA;
  int st;
  if (io.dk <= 64)
    st = io.dv <= 64 ? launch_sizes<64, 64>(tm, a, s) : launch_sizes<64, 128>(tm, a, s);
  else
    st = io.dv <= 64 ? launch_sizes<128, 64>(tm, a, s) : launch_sizes<128, 128>(tm, a, s);
  if (!pad || st != SDM_OK) return st;
  const long long rows = (long long)io.B * io.T * io.H, blocks = (rows + kPadThreads / 32 * kPadRows - 1) / (kPadThreads / 32 * kPadRows);
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kPadThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, narrow_kernel, static_cast<const __nv_bfloat16*>(io.o), rows, io.dv, dv,
                         static_cast<__nv_bfloat16*>(given.o)) != cudaSuccess)
    return SDM_ECUDA;
  return last_launch_status();
}

}  // namespace sdm
