// Selective state space scan, over prompts and for single tokens.
//
//   delta_t[d] = softplus(dt_t[d] + dt_bias[d])            (softplus optional)
//   h_t[d,n]   = exp(delta_t[d] A[d,n]) h_{t-1}[d,n] + delta_t[d] x_t[d] B_t[g,n]
//   y_t[d]     = (sum_n C_t[g,n] h_t[d,n] + D[d] x_t[d]) silu(z_t[d])
//
// with channel d in group g = d / (Dm / G).  Everything is computed and held in fp32; inputs and
// y are bf16 or fp32.
//
// Each (t, d, n) costs one exp2 and four fp32 operations (two products, two fused multiply-adds).
// A GB300 SM does 32 exp2 and 31 such foursomes a clock (measured), so with N = 16 and bf16 the
// arithmetic takes 1.5 times as long as HBM does for the 8 bytes of an element: the arithmetic is
// what has to be kept fed.  16 x 2048 x 4096 x 16 bf16 takes 0.69 ms, a third of the exp2 rate: 121
// instructions for 512 (t, d, n), 81 of them in the recurrence, at 67 % issue.  Two of an
// instruction's operations are packed in the input product and the read-out; packing the exponent's
// product costs more in moves than it saves (a loop of its own: 98 clocks a warp and 512 (t, d, n)
// so, 115 with all of it packed, 102 with none).
#include <type_traits>

#include "sdm_layers.cuh"

namespace sdm {
namespace {

constexpr int kThreads = 128;
constexpr int kLaneStates = 8;  // states a lane holds of each of its channels, at most
constexpr int kTokenThreads = 64;
constexpr int token_rows(int lanes) { return lanes < 2 ? 1 : 2; }  // sequences a lane works on
constexpr int kTT = 16;       // tokens of a shared-memory tile
constexpr int kMinChunk = 32; // tokens of a chunk, at least
constexpr int kSteps = 4;     // tokens taken together by a lane

struct ScanArgs {
  sdm_ssm_args io;
  int tiles_g, Dg;             // channel tiles of a group (one token: of a row), channels of a group
  int chunks, chunk;           // chunks of a sequence, tokens of a chunk (a multiple of kTT)
  float* ws_h;                 // [chunks][B][Dm][ws_n]: state before chunk 0, then each chunk's own end
  float* ws_d;                 // [chunks][B][Dm]: sum of delta over each chunk
  int ws_n;                    // N up to a multiple of 4
  bool vec_s;                  // rows of A and of the states start on 16 bytes
  bool vec;                    // rows of x, dt, z and y in 16-byte pieces; one token: four states a word
  bool vec_bc;                 // rows of B and C in 16-byte pieces; one token: four entries a word
  int* dev_err;
};

// A in units of exp2, finite, so that a step of size 0 has the decay 1 (0 times an infinite rate
// would have none).
__device__ __forceinline__ float decay_rate(float A) {
  const float r = A * kLog2e;
  return r == r ? fminf(fmaxf(r, -3.402823466e38f), 3.402823466e38f) : r;  // NaN stays
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory, zeros where !in.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  const int n = in ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
// exp(delta A), with the rate in units of exp2.  The fast exp2 is low by 1.4e-8 of its value in the
// mean over arguments from -1/8 to -1/256 (measured; 6e-9 nearer 0), and a slowly decaying state
// collects that over as many tokens as it remembers: the end state of 8192 tokens was off by 4.2e-7,
// 2.1e-7 with the mean added to the exponent, where it costs nothing.  A step of size 0 still has the
// decay 1: 2e-8 is under half a unit in the last place.
__device__ __forceinline__ float decay(float delta, float rate) {
  return exp2_fast(fmaf(delta, rate, 2.0e-8f));
}

// A state carried over a chunk that adds `end` to it: exp(sum A) h + end.  Where the state grows, the
// factor may pass the largest float although its product with h, and each token's own factor, do
// not: it is then applied in two halves, and a state of 0 stays 0.
__device__ __forceinline__ float carried_up(float h, float sum, float rate, float end) {
  const float e = fmaf(sum, rate, 2.0e-8f);
  if (!(e > 64.0f)) return fmaf(exp2_fast(e), h, end);
  const float half = exp2_fast(0.5f * e);
  return h == 0.0f ? end : fmaf(half, half * h, end);
}

// One element where rows are not aligned to 16 bytes: 4 bytes are copied like 16, 2 bytes are loaded.
__device__ __forceinline__ void copy1(float* dst, const float* src, bool in) {
  const int n = in ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void copy1(__nv_bfloat16* dst, const __nv_bfloat16* src, bool in) {
  *dst = in ? *src : __nv_bfloat16(0.f);
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Four elements of a row: as they lie in memory (one word where VEC says that they are aligned to
// it, else the first n one by one), and as numbers.
template <typename T, bool VEC>
struct Four {
  uint32_t w[sizeof(T)];  // 4 sizeof(T) bytes
  __device__ void load(const T* p, int n) {
    if constexpr (VEC && sizeof(T) == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (VEC) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      T* e = reinterpret_cast<T*>(w);
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = j < n ? p[j] : T(0.f);
    }
  }
  // The same for what is read once: L2 keeps other lines before it.
  __device__ void load_once(const T* p, int n) {
    if constexpr (VEC && sizeof(T) == 4) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      load(p, n);
    }
  }
  __device__ void clear() {
#pragma unroll
    for (int j = 0; j < int(sizeof(T)); ++j) w[j] = 0;
  }
  __device__ float operator[](int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
  }
};

// Passes over a sequence: one block takes all tokens (kWhole); or the sequence is cut in chunks,
// every chunk but the last is reduced to its end state from zero and its sum of delta (kReduce), and
// each chunk then starts from the given state carried through those before it (kJoin).  Chunks
// share A, so a chunk decays the state by exp(A sum(delta)).  The first pass also copies the given
// state, so that the second may write the new one in its place.
enum Pass { kWhole = 0, kReduce = 1, kJoin = 2 };

// L lanes share a channel, N states each; a lane has a pair of channels.
template <typename T, int L, int N>
struct Tile {
  static constexpr int V = Piece<T>::n;
  static constexpr int CH = 2 * kThreads / L;       // channels of a block
  static constexpr int NP = L * N;                  // padded number of states
  static constexpr int RV = CH / V;                 // pieces of a tile row
  static constexpr int pieces = kTT * RV;           // pieces of a tile
  static constexpr int raw = kTT * CH * int(sizeof(T));
  static constexpr int raw_bc = kTT * NP * int(sizeof(T));
  static constexpr int stage = 3 * raw + 2 * raw_bc;        // x, dt, z, B, C as they come
  static constexpr int off_dx = 2 * stage;                  // {delta, delta, delta x, delta x} by pair
  static constexpr int off_b = off_dx + kTT * CH * 8;
  static constexpr int off_c = off_b + kTT * NP * 4;
  static constexpr int bytes = off_c + kTT * NP * 4;
};

// Four blocks an SM, so 128 registers a thread: left to itself the compiler stops at 96 (five blocks),
// and 16 x 2048 x 4096 x 16 takes 707 us instead of 685; with 168 (three blocks) 750.  Four is what a
// full card gives each SM with more than 8 states in bf16 and more than 16 in fp32; the other
// instances' tiles leave shared memory for fewer: fp32 with 9 to 16 states 3 blocks (71,680 bytes
// each), bf16 with up to 8 states 2 (83,968), fp32 with up to 8 states 1 (134,144).
template <typename T, int L, int kS, int PASS>
__global__ void __launch_bounds__(kThreads, 4) scan_kernel(const __grid_constant__ ScanArgs a) {
  using S = Tile<T, L, kS>;
  constexpr int V = S::V;
  extern __shared__ __align__(16) uint8_t smem[];
  if (PASS == kReduce) allow_next();
  if (PASS == kJoin) wait_previous();
  const sdm_ssm_args& io = a.io;
  const int tid = threadIdx.x;

  // block -> (channel tile, sequence, chunk)
  int id = blockIdx.x;
  const int nct = a.tiles_g * io.G;
  const int ct = id % nct;
  id /= nct;
  const int b = id % io.B;
  const int chunk = PASS == kWhole ? 0 : id / io.B;
  const int g = ct / a.tiles_g;
  const int c0 = (ct - g * a.tiles_g) * S::CH;  // first channel of the tile in its group
  const int d0 = g * a.Dg + c0;
  const int nch = min(S::CH, a.Dg - c0);

  const int slot = row_slot(io.slots, b, io.n_slots, a.dev_err);
  const int len = slot < 0 ? 0 : row_length(io.lengths, b, io.T);
  const int t_lo = PASS == kWhole ? 0 : chunk * a.chunk;
  const int t_hi = PASS == kWhole ? io.T : min(t_lo + a.chunk, io.T);
  const int t_end = min(len, t_hi);  // tokens of this block that exist: [t_lo, t_end)

  const T* gx = static_cast<const T*>(io.x) + b * io.x_bs + d0;
  const T* gdt = static_cast<const T*>(io.dt) + b * io.dt_bs + d0;
  const T* gz = static_cast<const T*>(io.z) + (io.z ? b * io.z_bs + d0 : 0);
  const T* gB = static_cast<const T*>(io.Bm) + b * io.B_bs + g * io.N;
  const T* gC = static_cast<const T*>(io.Cm) + b * io.C_bs + g * io.N;
  T* gy = static_cast<T*>(io.y) + (size_t(b) * io.T) * io.Dm + d0;

  auto raw = [&](int st, int which) { return reinterpret_cast<T*>(smem + st * S::stage + which * S::raw); };
  auto raw_bc = [&](int st, int which) {
    return reinterpret_cast<T*>(smem + st * S::stage + 3 * S::raw + which * S::raw_bc);
  };
  float4* dx = reinterpret_cast<float4*>(smem + S::off_dx);
  float* sB = reinterpret_cast<float*>(smem + S::off_b);
  float* sC = reinterpret_cast<float*>(smem + S::off_c);

  auto load_tile = [&](int st, int t0) {
    const int nt = min(kTT, t_end - t0);
    if (a.vec) {
      for (int v = tid; v < S::pieces; v += kThreads) {
        const int t = v / S::RV, c = (v % S::RV) * V;
        const bool in = t < nt && c < nch;
        const long long tt = in ? t0 + t : 0;
        const int cc = in ? c : 0;
        copy16(raw(st, 0) + v * V, gx + tt * io.x_ts + cc, in);
        copy16(raw(st, 1) + v * V, gdt + tt * io.dt_ts + cc, in);
        if (PASS != kReduce && io.z) copy16(raw(st, 2) + v * V, gz + tt * io.z_ts + cc, in);
      }
    } else {
#pragma unroll 4
      for (int e = tid; e < kTT * S::CH; e += kThreads) {
        const int t = e / S::CH, c = e % S::CH;
        const bool in = t < nt && c < nch;
        const long long tt = in ? t0 + t : 0;
        const int cc = in ? c : 0;
        copy1(raw(st, 0) + e, gx + tt * io.x_ts + cc, in);
        copy1(raw(st, 1) + e, gdt + tt * io.dt_ts + cc, in);
        if (PASS != kReduce && io.z) copy1(raw(st, 2) + e, gz + tt * io.z_ts + cc, in);
      }
    }
    constexpr int NV = S::NP / V;
    bool rows = false;
    if constexpr (NV > 0) rows = a.vec_bc;
    if (rows) {
      for (int v = tid; v < kTT * NV; v += kThreads) {
        const int t = v / (NV ? NV : 1), n = (v % (NV ? NV : 1)) * V;
        const bool in = t < nt && n < io.N;
        const long long tt = in ? t0 + t : 0;
        const int nn = in ? n : 0;
        copy16(raw_bc(st, 0) + v * V, gB + tt * io.B_ts + nn, in);
        if (PASS != kReduce) copy16(raw_bc(st, 1) + v * V, gC + tt * io.C_ts + nn, in);
      }
    } else {
#pragma unroll 4
      for (int e = tid; e < kTT * S::NP; e += kThreads) {
        const int t = e / S::NP, n = e % S::NP;
        const bool in = t < nt && n < io.N;
        const long long tt = in ? t0 + t : 0;
        const int nn = in ? n : 0;
        copy1(raw_bc(st, 0) + e, gB + tt * io.B_ts + nn, in);
        if (PASS != kReduce) copy1(raw_bc(st, 1) + e, gC + tt * io.C_ts + nn, in);
      }
    }
    copies_commit();
  };

  // kThreads is a multiple of RV, so a thread's pieces all hold the same channels: their constants
  // stay in registers.
  static_assert(kThreads % S::RV == 0, "a thread's pieces share their channels");
  const int pr = tid % S::RV, pc = pr * V;
  uint64_t bias[V / 2], skip[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float bv[2], sv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = pc + 2 * i + k;
      bv[k] = io.dt_bias && c < nch ? io.dt_bias[d0 + c] : 0.f;
      sv[k] = PASS != kReduce && io.D && c < nch ? io.D[d0 + c] : 0.f;
    }
    bias[i] = pack2(bv[0], bv[1]);
    skip[i] = pack2(sv[0], sv[1]);
  }

  // Piece v of a tile holds channels c .. c+V-1 of token t; its pairs i go to plane i, so that the
  // pieces of a warp write and its lane groups read consecutive 16-byte words.
  auto prepare_tile = [&](int st) {
    for (int v = tid; v < S::pieces; v += kThreads) {
      const int t = v / S::RV;
      float x[V], d[V];
      Piece<T>::load(*reinterpret_cast<const uint4*>(raw(st, 0) + v * V), x);
      Piece<T>::load(*reinterpret_cast<const uint4*>(raw(st, 1) + v * V), d);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        uint64_t dl = add2(pack2(d[2 * i], d[2 * i + 1]), bias[i]);
        if (io.softplus) dl = softplus2(dl);
        *reinterpret_cast<ulonglong2*>(&dx[t * (S::CH / 2) + i * S::RV + pr]) =
            make_ulonglong2(dl, mul2(dl, pack2(x[2 * i], x[2 * i + 1])));
      }
    }
    for (int v = tid; v < kTT * S::NP / 4; v += kThreads) {
      Four<T, true> f;
      f.load(raw_bc(st, 0) + 4 * v, 4);
      reinterpret_cast<float4*>(sB)[v] = make_float4(f[0], f[1], f[2], f[3]);
      if (PASS != kReduce) {
        f.load(raw_bc(st, 1) + 4 * v, 4);
        reinterpret_cast<float4*>(sC)[v] = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  };

  auto store_tile = [&](int st, int t0) {  // y of the tile out of dx
    const int nt = min(kTT, t_end - t0);
    for (int v = tid; v < S::pieces; v += kThreads) {
      const int t = v / S::RV;
      if (t >= nt || pc >= nch) continue;
      float x[V], o[V], z[V];
      Piece<T>::load(*reinterpret_cast<const uint4*>(raw(st, 0) + v * V), x);
      if (io.z) Piece<T>::load(*reinterpret_cast<const uint4*>(raw(st, 2) + v * V), z);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        uint64_t y = *reinterpret_cast<const uint64_t*>(&dx[t * (S::CH / 2) + i * S::RV + pr]);
        y = fma2(skip[i], pack2(x[2 * i], x[2 * i + 1]), y);
        if (io.z)
          y = mul2(mul2(y, pack2(z[2 * i], z[2 * i + 1])), pack2(sigmoid(z[2 * i]), sigmoid(z[2 * i + 1])));
        unpack2(y, o[2 * i], o[2 * i + 1]);
      }
      T* p = gy + size_t(t0 + t) * io.Dm + pc;
      if (a.vec) {
        *reinterpret_cast<uint4*>(p) = Piece<T>::pack(o);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (pc + i < nch) from_f32(o[i], p + i);
      }
    }
  };

  // This lane's channels and states.
  const int sub = tid % L, pair = tid / L;
  const int ch = (pair % S::RV) * V + 2 * (pair / S::RV);  // the pair's first channel in the tile
  float A[2][kS], h[2][kS], dsum[2] = {0.f, 0.f};
  const size_t per = size_t(io.B) * io.Dm, bd = size_t(b) * io.Dm + d0;  // channels; of a chunk, of this tile
  // This lane's states of a row that starts at p: words of four where `vec` says that rows start on
  // 16 bytes (those of the workspace always do), zeros past the last state.
  auto get = [&](const float* p, bool vec, float (&v)[kS]) {
#pragma unroll
    for (int j = 0; j < kS; j += 4) {
      const int n = sub * kS + j;
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
      if (vec) {
        if (n < io.N) w = *reinterpret_cast<const float4*>(p + n);
      } else {
        if (n < io.N) w.x = p[n];
        if (n + 1 < io.N) w.y = p[n + 1];
        if (n + 2 < io.N) w.z = p[n + 2];
        if (n + 3 < io.N) w.w = p[n + 3];
      }
      v[j] = w.x;
      v[j + 1] = n + 1 < io.N ? w.y : 0.f;
      v[j + 2] = n + 2 < io.N ? w.z : 0.f;
      v[j + 3] = n + 3 < io.N ? w.w : 0.f;
    }
  };
  auto put = [&](float* p, bool vec, const float (&v)[kS]) {
#pragma unroll
    for (int j = 0; j < kS; j += 4) {
      const int n = sub * kS + j;
      if (vec) {
        if (n < io.N) *reinterpret_cast<float4*>(p + n) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < io.N) p[n + i] = v[j + i];
      }
    }
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int c = ch + k;
#pragma unroll
    for (int j = 0; j < kS; ++j) A[k][j] = h[k][j] = 0.f;
    if (c < nch) {
      get(io.A + size_t(d0 + c) * io.N, a.vec_s, A[k]);
#pragma unroll
      for (int j = 0; j < kS; ++j) A[k][j] = decay_rate(A[k][j]);
      if (slot >= 0) {
        const float* given = io.state + (size_t(slot) * io.Dm + d0 + c) * io.N;
        if (PASS == kWhole && io.state) get(given, a.vec_s, h[k]);
        if (PASS == kJoin) get(a.ws_h + (bd + c) * a.ws_n, true, h[k]);
        if (PASS == kReduce && chunk == 0) {
          float v[kS];
#pragma unroll
          for (int j = 0; j < kS; ++j) v[j] = 0.f;
          if (io.state) get(given, a.vec_s, v);
          put(a.ws_h + (bd + c) * a.ws_n, true, v);
        }
      }
    }
  }
  if (PASS == kJoin && slot >= 0) {
    // Four chunks at a time: what they bring does not depend on the state, so it is asked for together.
    constexpr int kBatch = 4;
    bool grows = !io.softplus;  // steps may be negative
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < kS; ++j) grows = grows || A[k][j] > 0.0f;
    for (int q0 = 0; q0 < chunk; q0 += kBatch) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = min(ch + k, nch - 1);  // lanes past the last channel follow it, to no effect
        float sum[kBatch], end[kBatch][kS];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int q = q0 + i;
          sum[i] = 0.f;  // a chunk of none: decay 1, nothing added
#pragma unroll
          for (int j = 0; j < kS; ++j) end[i][j] = 0.f;
          if (q < chunk) {
            sum[i] = a.ws_d[q * per + bd + c];
            get(a.ws_h + ((q + 1) * per + bd + c) * a.ws_n, true, end[i]);
          }
        }
        if (grows) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int j = 0; j < kS; ++j) h[k][j] = carried_up(h[k][j], sum[i], A[k][j], end[i][j]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
          for (int j = 0; j < kS; ++j) h[k][j] = fmaf(decay(sum[i], A[k][j]), h[k][j], end[i][j]);
      }
    }
  }

  // G tokens from t of the prepared tile.  Their sums over the states are kept until the end and
  // added over the channel's lanes together, so that no token waits for the one before it.
  auto steps = [&](int t, auto count) {
    constexpr int G = decltype(count)::value;
    float y[G][2];
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const ulonglong2* pB = reinterpret_cast<const ulonglong2*>(sB + (t + s) * S::NP + sub * kS);
      const ulonglong2* pC = reinterpret_cast<const ulonglong2*>(sC + (t + s) * S::NP + sub * kS);
      const float4 w = dx[(t + s) * (S::CH / 2) + pair];
      const float dl[2] = {w.x, w.y};
      const uint64_t dlx[2] = {pack2(w.z, w.z), pack2(w.w, w.w)};
      uint64_t acc[2][2];
#pragma unroll
      for (int j = 0; j < kS / 4; ++j) {
        const ulonglong2 vB = pB[j];
        ulonglong2 vC;
        if (PASS != kReduce) vC = pC[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int q = 4 * j + 2 * i;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x0, x1;
            unpack2(mul2(dlx[k], i ? vB.y : vB.x), x0, x1);
            h[k][q] = fmaf(decay(dl[k], A[k][q]), h[k][q], x0);
            h[k][q + 1] = fmaf(decay(dl[k], A[k][q + 1]), h[k][q + 1], x1);
            if (PASS != kReduce) {
              const uint64_t hh = pack2(h[k][q], h[k][q + 1]), cc = i ? vC.y : vC.x;
              acc[k][i] = j ? fma2(hh, cc, acc[k][i]) : mul2(hh, cc);
            }
          }
        }
      }
      if (PASS == kReduce) {
        dsum[0] += w.x;
        dsum[1] += w.y;
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float y0, y1;
          unpack2(add2(acc[k][0], acc[k][1]), y0, y1);
          y[s][k] = y0 + y1;
        }
      }
    }
    if constexpr (PASS != kReduce) {
      // The sums replace the pair's delta words, which the channel's lanes alone read.
      float* out = reinterpret_cast<float*>(&dx[t * (S::CH / 2) + pair]);
      constexpr int row = 2 * S::CH;  // floats between tokens
      if constexpr (L == 1) {
#pragma unroll
        for (int s = 0; s < G; ++s) *reinterpret_cast<float2*>(out + s * row) = make_float2(y[s][0], y[s][1]);
      } else {
        // neighbours swap channels: an even lane goes on with channel 0, an odd one with channel 1
        float v[G];
#pragma unroll
        for (int s = 0; s < G; ++s) {
          const float give = sub & 1 ? y[s][0] : y[s][1], keep = sub & 1 ? y[s][1] : y[s][0];
          v[s] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
        }
        // then, as far as they go, lanes halve the tokens between them; the rest add all they have
        int n = G, first = 0;
#pragma unroll
        for (int o = 2; o < L; o *= 2) {
          if (n > 1) {
            n /= 2;
            const bool up = (sub & o) != 0;
#pragma unroll
            for (int s = 0; s < G / 2; ++s)
              if (s < n) {
                const float give = up ? v[s] : v[s + n], keep = up ? v[s + n] : v[s];
                v[s] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
              }
            if (up) first += n;
          } else {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
          }
        }
        if (L <= 2 * G || sub < 2 * G) {
#pragma unroll
          for (int s = 0; s < G; ++s)
            if (s < n) out[(first + s) * row + (sub & 1)] = v[s];
        }
      }
    }
  };

  if (t_lo < t_end) {
    load_tile(0, t_lo);
    copies_wait();
    __syncthreads();
    prepare_tile(0);
    if (t_lo + kTT < t_end) load_tile(1, t_lo + kTT);
    __syncthreads();
    int st = 0;
    for (int t0 = t_lo; t0 < t_end; t0 += kTT, st ^= 1) {
      const int nt = min(kTT, t_end - t0);
      int t = 0;
      for (; t + kSteps <= nt; t += kSteps) steps(t, std::integral_constant<int, kSteps>());
      for (; t < nt; ++t) steps(t, std::integral_constant<int, 1>());
      copies_wait();
      __syncthreads();
      if (PASS != kReduce) store_tile(st, t0);
      if (t0 + kTT < t_end) prepare_tile(st ^ 1);
      __syncthreads();
      if (t0 + 2 * kTT < t_end) load_tile(st, t0 + 2 * kTT);
    }
  }

  if (PASS != kReduce) {  // tokens past the sequence's length
    const int z0 = max(t_end, t_lo);
    const long long cells = (long long)(t_hi - z0) * nch;
    for (long long e = tid; e < cells; e += kThreads)
      from_f32(0.f, gy + size_t(z0 + e / nch) * io.Dm + int(e % nch));
  }
  const bool last = PASS == kWhole || (PASS == kJoin && chunk == a.chunks - 1);
  if (slot >= 0 && (PASS == kReduce || (last && io.state_out))) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = ch + k;
      if (c >= nch) continue;
      if (PASS == kReduce) {
        put(a.ws_h + ((chunk + 1) * per + bd + c) * a.ws_n, true, h[k]);
        if (sub == 0) a.ws_d[chunk * per + bd + c] = dsum[k];
      } else {
        put(io.state_out + (size_t(slot) * io.Dm + d0 + c) * io.N, a.vec_s, h[k]);
      }
    }
  }
}

// One token: a lane has 4 Q states of a channel in each of R sequences, L lanes a channel.  HBM bounds
// it, the states read and written once: R states are under way in every lane, everything that does
// not wait for a slot is asked for first, and what a channel computes once (step size, gate) is done
// for each sequence by one of its lanes, lane r < R for sequence r.  States pass once through L2,
// marked so (26.6 us a call at 256 x 4096 x 16 bf16 with slots, 0.79 of HBM's rate; 30.6 unmarked;
// blocks that stay and walk over the sequences took 46).  VEC: four states, and four entries of B and C, are a word.
template <typename T, int L, int Q, bool VEC>
__global__ void __launch_bounds__(kTokenThreads) token_kernel(const __grid_constant__ ScanArgs a) {
  constexpr int R = token_rows(L);
  const sdm_ssm_args& io = a.io;
  const int sub = threadIdx.x % L, own = sub % R;
  const int group = int(blockIdx.x) / a.tiles_g;  // of R sequences; tiles_g blocks hold its channels
  const int channel = (int(blockIdx.x) - group * a.tiles_g) * (kTokenThreads / L) + int(threadIdx.x) / L;
  const bool present = channel < io.Dm;  // lanes past the last channel only take part in the shuffles
  const int d = present ? channel : 0;
  const int b0 = group * R, rows = present ? min(R, io.B - b0) : 0;
  const int n0 = sub * 4 * Q;
  int left[Q];  // states of word q that exist
#pragma unroll
  for (int q = 0; q < Q; ++q) left[q] = io.N - n0 - 4 * q;
  const size_t at = size_t(d) * io.N + n0, row = size_t(io.Dm) * io.N;

  int slot[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
    slot[r] = r < rows ? row_slot(io.slots, b0 + r, io.n_slots, d == 0 && sub == 0 ? a.dev_err : nullptr) : -1;
  float x = 0.f, dl = 0.f, z = 0.f;
  if (own < rows) {
    const long long b = b0 + own;
    x = to_f32(static_cast<const T*>(io.x)[b * io.x_bs + d]);
    dl = to_f32(static_cast<const T*>(io.dt)[b * io.dt_bs + d]);
    if (io.z) z = to_f32(static_cast<const T*>(io.z)[b * io.z_bs + d]);
  }
  Four<float, VEC> A[Q], h4[R][Q];
  Four<T, VEC> B[R][Q], C[R][Q];
  const int bc = (io.G > 1 ? d / a.Dg * io.N : 0) + n0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    A[q].clear();
    if (left[q] > 0) A[q].load(io.A + at + 4 * q, left[q]);
    const T* pB = static_cast<const T*>(io.Bm) + b0 * io.B_bs + bc + 4 * q;
    const T* pC = static_cast<const T*>(io.Cm) + b0 * io.C_bs + bc + 4 * q;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      B[r][q].clear();
      C[r][q].clear();
      if (r < rows && left[q] > 0) {
        B[r][q].load(pB, left[q]);
        C[r][q].load(pC, left[q]);
      }
      pB += io.B_bs;
      pC += io.C_bs;
    }
  }
  const float bias = io.dt_bias ? io.dt_bias[d] : 0.f, skip = io.D ? io.D[d] : 0.f;
  bool live[R], mine = false;  // the sequence has a state and a token
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float* p = io.state + at + size_t(unsigned(max(slot[r], 0))) * row;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      h4[r][q].clear();
      if (slot[r] >= 0 && io.state && left[q] > 0) h4[r][q].load_once(p + 4 * q, left[q]);
    }
    live[r] = slot[r] >= 0 && row_length(io.lengths, b0 + r, 1) > 0;
    mine = mine || (own == r && live[r]);
  }

  dl += bias;
  if (io.softplus) dl = softplus(dl);
  const float dlx = dl * x;
  float rate[Q][4], y[R];
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int j = 0; j < 4; ++j) rate[q][j] = decay_rate(A[q][j]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float dr = __shfl_sync(0xFFFFFFFFu, dl, r, L), dx = __shfl_sync(0xFFFFFFFFu, dlx, r, L);
    float* p = io.state_out + at + size_t(unsigned(max(slot[r], 0))) * row;
    const bool keep = slot[r] >= 0 && io.state_out;
    y[r] = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = h4[r][q][j];
        if (live[r]) {
          h[j] = fmaf(decay(dr, rate[q][j]), h[j], dx * B[r][q][j]);
          y[r] = fmaf(h[j], C[r][q][j], y[r]);
        }
      }
      if (keep && left[q] > 0) {
        if constexpr (VEC) {
          __stcs(reinterpret_cast<float4*>(p + 4 * q), make_float4(h[0], h[1], h[2], h[3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < left[q]) p[4 * q + j] = h[j];
        }
      }
    }
  }
  // Sums over the channel's lanes; lane r keeps sequence r's.
  if constexpr (R == 2) {
    const bool odd = sub & 1;
    const float give = odd ? y[0] : y[1], keep = odd ? y[1] : y[0];
    y[0] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, 1);
#pragma unroll
    for (int o = 2; o < L; o *= 2) y[0] += __shfl_xor_sync(0xFFFFFFFFu, y[0], o);
  }
  if (sub < R && own < rows) {
    float v = fmaf(skip, x, y[0]);
    if (io.z) v *= silu(z);
    from_f32(mine ? v : 0.f, static_cast<T*>(io.y) + size_t(b0 + own) * io.Dm + d);
  }
}

int lanes_for(int N, int per) {
  int l = 1;
  while (l * per < N) l *= 2;
  return l;
}

template <typename T, int L, int S, int PASS>
int launch_pass(const ScanArgs& a, int chunks, cudaStream_t s) {
  constexpr int bytes = Tile<T, L, S>::bytes;
  auto fn = scan_kernel<T, L, S, PASS>;
  static PerDevice ready;
  if (ready.get([&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? 0 : -1;
      }) < 0)
    return SDM_ECUDA;
  const long long blocks = (long long)a.tiles_g * a.io.G * a.io.B * chunks;
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PASS == kJoin ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

template <typename T, int L, int S>
int launch_passes(ScanArgs& a, cudaStream_t s) {
  a.tiles_g = (a.Dg + Tile<T, L, S>::CH - 1) / Tile<T, L, S>::CH;
  if (a.chunks <= 1) return launch_pass<T, L, S, kWhole>(a, 1, s);
  const int st = launch_pass<T, L, S, kReduce>(a, a.chunks - 1, s);
  return st != SDM_OK ? st : launch_pass<T, L, S, kJoin>(a, a.chunks, s);
}

template <typename T>
int launch_scan(ScanArgs& a, cudaStream_t s) {
  if (a.io.N <= 4) return launch_passes<T, 1, 4>(a, s);
  switch (lanes_for(a.io.N, kLaneStates)) {
    case 1: return launch_passes<T, 1, kLaneStates>(a, s);
    case 2: return launch_passes<T, 2, kLaneStates>(a, s);
    case 4: return launch_passes<T, 4, kLaneStates>(a, s);
    case 8: return launch_passes<T, 8, kLaneStates>(a, s);
    case 16: return launch_passes<T, 16, kLaneStates>(a, s);
    default: return SDM_EUNSUPPORTED;
  }
}

template <typename T, int L, int Q>
int launch_token_l(ScanArgs& a, cudaStream_t s) {
  constexpr int R = token_rows(L), channels = kTokenThreads / L;
  a.tiles_g = (a.io.Dm + channels - 1) / channels;
  const long long blocks = (long long)((a.io.B + R - 1) / R) * a.tiles_g;
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  if (a.vec && a.vec_bc)
    token_kernel<T, L, Q, true><<<unsigned(blocks), kTokenThreads, 0, s>>>(a);
  else
    token_kernel<T, L, Q, false><<<unsigned(blocks), kTokenThreads, 0, s>>>(a);
  return last_launch_status();
}

template <typename T>
int launch_token(ScanArgs& a, cudaStream_t s) {
  if (a.io.N <= 4) return launch_token_l<T, 1, 1>(a, s);
  switch (lanes_for(a.io.N, 8)) {
    case 1: return launch_token_l<T, 1, 2>(a, s);
    case 2: return launch_token_l<T, 2, 2>(a, s);
    case 4: return launch_token_l<T, 4, 2>(a, s);
    case 8: return launch_token_l<T, 8, 2>(a, s);
    case 16: return launch_token_l<T, 16, 2>(a, s);
    default: return SDM_EUNSUPPORTED;
  }
}

// Chunks of a sequence and tokens of a chunk: one chunk where the channels alone give the card 208
// blocks, else as many as keep within four blocks an SM, of kMinChunk tokens at least.  A block's
// tokens wait on one another, so an SM with two blocks takes little longer than with one (2048
// tokens, 4096 channels a sequence: 343, 397, 560 and 685 us with one to four), and two passes cost
// 1.5 times the arithmetic of one: 128 blocks take 275 us in four chunks and 343 in one, 192 blocks
// 380 and 397, 256 blocks 515 and 397.  Four blocks an SM against three: 32768 tokens of 2048
// channels 554 us against 627 (512 now); chunks of 32 tokens against 64: 512 tokens of 1024 channels
// 28.5 us against 31.3.
//
// All of that is bf16 with 16 states, and the two numbers stand for every type and state count although
// instances with fewer blocks an SM would cut later: fp32 with 8 states, a block an SM, takes 587 us for 9 sequences
// of 2048 x 4096 (cut) and 792 for 13 (not cut, two rounds of 396).  Nor is the join in the rule, whose
// blocks walk all chunks before theirs: 32,768 tokens of 64 channels, 512 chunks, take 304 us, of 256
// channels 245.
void cut(int B, int T, int Dm, int N, int G, int* chunks, long long* chunk) {
  const int L = lanes_for(N, kLaneStates), CH = 2 * kThreads / L;
  const long long blocks = (long long)B * G * (((long long)Dm / G + CH - 1) / CH);
  long long n = blocks >= 208 ? 1 : 608 / blocks;
  n = n < T / kMinChunk ? n : T / kMinChunk;
  if (n < 1) n = 1;
  const long long per = ((T + n - 1) / n + kTT - 1) / kTT * kTT;
  *chunk = per;
  *chunks = T > 0 ? int((T + per - 1) / per) : 1;
}

bool sizes_ok(int B, int T, int Dm, int N, int G) {
  return B >= 1 && T >= 0 && Dm >= 1 && N >= 1 && G >= 1 && Dm % G == 0;
}

// Whether y, the new states or the workspace overlap anything else of the call.  The state may be
// updated in place, and y may be x, dt or z: a block reads of these only the tokens and channels whose
// y it writes, a tile into shared memory before that tile's y; the pass that reduces chunks is over
// when the first y is written.
bool overlap(const sdm_ssm_args& io, const void* workspace, size_t workspace_bytes) {
  const long long es = io.dtype == SDM_F32 ? 4 : 2, row = io.Dm * es, bc = (long long)io.G * io.N * es;
  const long long sn = 4LL * io.n_slots * io.Dm * io.N, yn = (long long)io.B * io.T * row, wn = (long long)workspace_bytes;
  auto rows = [&](const void* p, long long bs, long long ts, long long bytes) {
    return Extent{p, io.B, bs * es, io.T, ts * es, bytes};
  };
  auto like_y = [&](const Extent& e) {
    return e.p == io.y && (io.B == 1 || e.s1 == io.T * row) && (io.T == 1 || e.s2 == row);
  };
  const Extent state = dense(io.state, sn), y = dense(io.y, yn);
  for (const Extent& e : {rows(io.x, io.x_bs, io.x_ts, row), rows(io.dt, io.dt_bs, io.dt_ts, row),
                          rows(io.z, io.z_bs, io.z_ts, row)})
    if ((!like_y(e) && meets(e, io.y, yn)) || meets(e, io.state_out, sn) || meets(e, workspace, wn)) return true;
  for (const Extent& e : {rows(io.Bm, io.B_bs, io.B_ts, bc), rows(io.Cm, io.C_bs, io.C_ts, bc),
                          dense(io.A, 4LL * io.Dm * io.N), dense(io.D, 4LL * io.Dm), dense(io.dt_bias, 4LL * io.Dm),
                          dense(io.lengths, 4LL * io.B), dense(io.slots, 4LL * io.B)})
    if (meets(e, io.y, yn) || meets(e, io.state_out, sn) || meets(e, workspace, wn)) return true;
  return (io.state != io.state_out && meets(state, io.state_out, sn)) || meets(state, io.y, yn) ||
         meets(state, workspace, wn) || meets(y, io.state_out, sn) || meets(y, workspace, wn) ||
         meets(dense(io.state_out, sn), workspace, wn);
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t sdm_selective_scan_workspace_size(int B, int T, int Dm, int N, int G) {
  if (!sizes_ok(B, T, Dm, N, G) || N > SDM_MAX_SSM_N) return 0;
  int chunks;
  long long chunk;
  cut(B, T, Dm, N, G, &chunks, &chunk);
  if (chunks <= 1) return 0;
  return size_t(chunks) * B * Dm * ((N + 3) / 4 * 4 + 1) * 4;
}

extern "C" int sdm_selective_scan(const sdm_ssm_args* args, void* workspace, size_t workspace_bytes,
                                  int* dev_err, void* stream) {
  if (!args) return SDM_EINVAL;
  const sdm_ssm_args& io = *args;
  if (!sizes_ok(io.B, io.T, io.Dm, io.N, io.G) || bad_dtype(io.dtype)) return SDM_EINVAL;
  if (io.N > SDM_MAX_SSM_N || (long long)io.B * io.T > 0x7FFFFFFFLL || io.Dm > 0x3FFFFFF)
    return SDM_EUNSUPPORTED;
  int chunks;
  long long chunk;
  cut(io.B, io.T, io.Dm, io.N, io.G, &chunks, &chunk);
  // A token's index may run past the last chunk's end by two tiles, and stays an int.
  if (chunks * chunk > 0x7FFFFFFFLL - 2 * kTT) return SDM_EUNSUPPORTED;
  if ((io.state || io.state_out || io.slots) && io.n_slots < (io.slots ? 1 : io.B)) return SDM_EINVAL;
  const uintptr_t odd = io.dtype == SDM_F32 ? 3 : 1;
  auto off = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (!io.A || off(io.A, 3) || off(io.D, 3) || off(io.dt_bias, 3) || off(io.state, 3) ||
      off(io.state_out, 3) || off(io.lengths, 3) || off(io.slots, 3) || off(dev_err, 3))
    return SDM_EALIGN;
  if (io.T > 0 && (!io.x || !io.dt || !io.Bm || !io.Cm || !io.y || off(io.x, odd) || off(io.dt, odd) ||
                   off(io.Bm, odd) || off(io.Cm, odd) || off(io.z, odd) || off(io.y, odd)))
    return SDM_EALIGN;
  if (io.T == 0 && (io.state == io.state_out || !io.state_out)) return SDM_OK;

  ScanArgs a = {};
  a.io = io;
  a.Dg = io.Dm / io.G;
  a.dev_err = dev_err;
  cudaStream_t s = as_stream(stream);
  if (io.T == 1) {
    if (overlap(io, nullptr, 0)) return SDM_EOVERLAP;
    // Four states a word, and four entries of B and C (8 bytes of bf16, 16 of fp32).
    const uintptr_t word = io.dtype == SDM_F32 ? 15 : 7;
    a.vec = io.N % 4 == 0 && !off(io.A, 15) && !off(io.state, 15) && !off(io.state_out, 15);
    a.vec_bc = io.N % 4 == 0 && io.B_bs % 4 == 0 && io.C_bs % 4 == 0 && !off(io.Bm, word) && !off(io.Cm, word);
    return io.dtype == SDM_F32 ? launch_token<float>(a, s) : launch_token<__nv_bfloat16>(a, s);
  }
  const size_t need = sdm_selective_scan_workspace_size(io.B, io.T, io.Dm, io.N, io.G);
  a.chunks = chunks;
  a.chunk = int(chunk);
  if (need) {
    if (!aligned16(workspace)) return SDM_EALIGN;
    if (workspace_bytes < need) return SDM_ENOSPACE;
    a.ws_n = (io.N + 3) / 4 * 4;
    a.ws_h = static_cast<float*>(workspace);
    a.ws_d = a.ws_h + size_t(a.chunks) * io.B * io.Dm * a.ws_n;
  }
  if (overlap(io, need ? workspace : nullptr, need)) return SDM_EOVERLAP;
  const int V = io.dtype == SDM_F32 ? 4 : 8;
  auto rows16 = [&](const void* p, long long bs, long long ts) {
    return !p || (!off(p, 15) && bs % V == 0 && ts % V == 0);
  };
  a.vec = a.Dg % V == 0 && rows16(io.x, io.x_bs, io.x_ts) && rows16(io.dt, io.dt_bs, io.dt_ts) &&
          rows16(io.z, io.z_bs, io.z_ts) && !off(io.y, 15);
  a.vec_s = io.N % 4 == 0 && !off(io.A, 15) && !off(io.state, 15) && !off(io.state_out, 15);
  a.vec_bc = io.N % V == 0 && rows16(io.Bm, io.B_bs, io.B_ts) && rows16(io.Cm, io.C_bs, io.C_ts);
  return io.dtype == SDM_F32 ? launch_scan<float>(a, s) : launch_scan<__nv_bfloat16>(a, s);
}
