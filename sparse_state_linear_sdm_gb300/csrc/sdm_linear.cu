// Linear attention with a decay for each head, over prompts and for single tokens.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,   S [dk, dv] in fp32
//
// Three forms.  A single token streams the states through once (token_kernel; HBM bounds it).  Prompts
// take their tokens one after the other with the state in registers (step_kernel: any type, alignment
// and size), or, in bf16 with dk up to 128, in chunks of 128 tokens on the tensor cores (sdm_linear_tiles.cu; rows that
// TMA cannot take are copied first where dk or dv is at fault, and taken one by one where only strides are).
//
// One token of 256 sequences, 16 heads of 128 x 128 in slots: 83 us, 0.96 of the HBM floor.  step_kernel is bound by its two
// multiply-adds a state and token, which one block an SM leaves at half of their rate (8 x 2048 x 16 heads of 128 in fp32:
// 665 us, floor 230; two tokens at a time 727 of 690).
//
// Where sequences and heads leave the card short, a sequence is cut into segments: every segment but the last
// is reduced to its end state from zero and its sum of g, a small kernel turns those into the state in front of each
// segment, and every segment then runs from there: up to twice the work, side by side.
#include "sdm_linear.cuh"

namespace sdm {
namespace {

constexpr int kStepTokens = 16;  // tokens of a shared-memory tile
constexpr int kRows = 16;        // state rows of a lane
constexpr int kCols = 4;         // and columns
constexpr int kStepWarps = 8;    // of a block, at most

// A warp holds a DK x cols piece of a state: R lanes share the rows, 32 / R groups of lanes have four columns each.  (With
// eight, a head of 128 x 128 is four warps, one for each scheduler of an SM: 779 us instead of 690.)
template <int DK>
struct Warp {
  static constexpr int R = DK / kRows;
  static constexpr int cols = 32 / R * kCols;
};

// Shared memory of a block: two tiles as they come (q, k and the block's columns of v of 16 tokens, and g), the
// tile as floats where it comes as bf16, and o.
template <typename T, int DK>
struct StepTile {
  int vc, row, raw, off_f, off_o, bytes;
  __host__ __device__ explicit StepTile(int warps) {
    vc = warps * Warp<DK>::cols;
    row = 2 * DK + vc;
    raw = kStepTokens * row * int(sizeof(T)) + kStepTokens * 4;
    off_f = 2 * raw;
    off_o = off_f + (sizeof(T) == 4 ? 0 : kStepTokens * row * 4);
    bytes = off_o + kStepTokens * vc * 4;
  }
};

// Within a tile the state is held as S = e^{G_t} s, G_t the sum of g from the tile's start: a token then costs
// s += (e^{-G_t} v) k^T and o = e^{G_t} q s, two multiply-adds a state instead of three, and a slow decay is not
// rounded at every token.  Where |G_t| passes kLazy within a tile, its tokens decay s one by one instead.  The sums are
// carried in two floats, and the exponential takes both (in one, 4,000 tokens at 0.001 left 4e-6).
constexpr float kLazy = 30.f;

struct TwoSum {
  float hi, lo;
  __device__ __forceinline__ TwoSum operator+(const TwoSum& o) const {
    const float s = hi + o.hi, z = s - hi;
    return {s, (lo + o.lo) + ((hi - (s - z)) + (o.hi - z))};
  }
  __device__ __forceinline__ TwoSum from_lane(int lane) const {
    return {__shfl_sync(0xFFFFFFFFu, hi, lane & 31), __shfl_sync(0xFFFFFFFFu, lo, lane & 31)};
  }
  // e^(hi + lo): what the argument's rounding leaves is multiplied on.
  __device__ __forceinline__ float exp(float sign) const {
    // 1.9259630e-8: what kLog2e leaves of log2 e.
    const float x = hi * kLog2e, rest = fmaf(hi, kLog2e, -x) + fmaf(hi, 1.925963033500e-8f, lo * kLog2e);
    const float e = exp2_fast(sign * x);
    return fmaf(e, sign * 0.69314718f * rest, e);
  }
};

template <typename T, int DK, int PASS>
__global__ void __launch_bounds__(32 * kStepWarps, 2) step_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int R = Warp<DK>::R, CW = Warp<DK>::cols, V = Piece<T>::n;
  extern __shared__ __align__(16) uint8_t smem[];
  const sdm_linear_args& io = a.io;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads / 32;
  const StepTile<T, DK> lay(warps);
  if (PASS == kReduce) allow_next();
  if (PASS == kJoin) wait_previous();

  const Place p = place_of<PASS>(a);
  const int c0 = p.vt * lay.vc;              // first column of the block
  const int nv = min(lay.vc, io.dv - c0);
  const int warp = tid >> 5, lane = tid & 31, r = lane % R;
  const int col = warp * CW + lane / R * kCols;  // this lane's first column in the block
  const int dk = io.dk;

  const T* gq = static_cast<const T*>(io.q) + p.b * io.q_bs + (long long)p.hk * dk;
  const T* gk = static_cast<const T*>(io.k) + p.b * io.k_bs + (long long)p.hk * dk;
  const T* gv = static_cast<const T*>(io.v) + p.b * io.v_bs + (long long)p.h * io.dv + c0;
  const float* gg = io.g ? io.g + p.b * io.g_bs + p.h : nullptr;
  T* go = static_cast<T*>(io.o) + ((long long)p.b * io.T * io.H + p.h) * io.dv + c0;
  const long long ots = (long long)io.H * io.dv;

  auto raw = [&](int st) { return reinterpret_cast<T*>(smem + st * lay.raw); };
  auto raw_g = [&](int st) { return reinterpret_cast<float*>(smem + (st + 1) * lay.raw) - kStepTokens; };
  float* so = reinterpret_cast<float*>(smem + lay.off_o);

  auto load_tile = [&](int st, int t0) {
    const int nt = min(kStepTokens, p.t_end - t0);
    T* dst = raw(st);
    if (a.vec_qk) {
      constexpr int NP = DK / V;
      for (int e = tid; e < kStepTokens * 2 * NP; e += threads) {
        const int t = e / (2 * NP), w = e % (2 * NP), c = w % NP * V;
        const bool in = t < nt && c < dk, key = w >= NP;
        if (key || PASS != kReduce)
          copy16(dst + t * lay.row + (key ? DK : 0) + c,
                 (key ? gk : gq) + (in ? (t0 + t) * (key ? io.k_ts : io.q_ts) + c : 0), in);
      }
    } else {  // a token a warp
#pragma unroll 2
      for (int t = warp; t < kStepTokens; t += warps) {
        const int row = t0 + min(t, nt - 1);
        const T *rq = gq + row * io.q_ts, *rk = gk + row * io.k_ts;
#pragma unroll
        for (int c = lane; c < DK; c += 32) {
          const bool in = t < nt && c < dk;
          const int at = in ? c : 0;
          if (PASS != kReduce) copy1(dst + t * lay.row + c, rq + at, in);
          copy1(dst + t * lay.row + DK + c, rk + at, in);
        }
      }
    }
    if (a.vec_v) {
      const int NP = lay.vc / V;
      for (int e = tid; e < kStepTokens * NP; e += threads) {
        const int t = e / NP, c = e % NP * V;
        const bool in = t < nt && c < nv;
        copy16(dst + t * lay.row + 2 * DK + c, gv + (in ? (t0 + t) * io.v_ts + c : 0), in);
      }
    } else {
#pragma unroll 2
      for (int t = warp; t < kStepTokens; t += warps) {
        const T* rv = gv + (t0 + min(t, nt - 1)) * io.v_ts;
        for (int c = lane; c < lay.vc; c += 32) {
          const bool in = t < nt && c < nv;
          copy1(dst + t * lay.row + 2 * DK + c, rv + (in ? c : 0), in);
        }
      }
    }
    if (tid < kStepTokens) {
      if (gg && tid < nt)
        copy1(raw_g(st) + tid, gg + (t0 + tid) * io.g_ts, true);
      else
        raw_g(st)[tid] = 0.f;
    }
    copies_commit();
  };

  // This lane's rows: 4 r + 4 R i + 0 .. 3, i = 0 .. 3, so that the lanes of a group read consecutive words; s[i][c]
  // holds rows in pairs.
  uint64_t s[kRows / 2][kCols];
  auto row_of = [&](int i) { return 4 * r + 4 * R * (i / 2) + 2 * (i % 2); };
  const long long sn = (long long)dk * io.dv;
  const bool words = a.vec_s;
  auto read_state = [&](const float* src) {
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      float x[2][kCols];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = row_of(i) + j;
        const float* f = src + (long long)row * io.dv + c0 + col;
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < dk && words) {
            if (col + c < nv) w = *reinterpret_cast<const float4*>(f + c);
          } else if (row < dk) {
            if (col + c < nv) w.x = f[c];
            if (col + c + 1 < nv) w.y = f[c + 1];
            if (col + c + 2 < nv) w.z = f[c + 2];
            if (col + c + 3 < nv) w.w = f[c + 3];
          }
          x[j][c] = w.x, x[j][c + 1] = w.y, x[j][c + 2] = w.z, x[j][c + 3] = w.w;
        }
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c) s[i][c] = pack2(x[0][c], x[1][c]);
    }
  };
  auto write_state = [&](float* dst, float f) {
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      float x[2][kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) unpack2(s[i][c], x[0][c], x[1][c]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = row_of(i) + j;
        if (row >= dk) continue;
        float* d = dst + (long long)row * io.dv + c0 + col;
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          if (words) {
            if (col + c < nv)
              *reinterpret_cast<float4*>(d + c) = make_float4(x[j][c] * f, x[j][c + 1] * f, x[j][c + 2] * f, x[j][c + 3] * f);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (col + c + k < nv) d[c + k] = x[j][c + k] * f;
          }
        }
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kRows / 2; ++i)
#pragma unroll
    for (int c = 0; c < kCols; ++c) s[i][c] = 0;
  const long long bh = (long long)p.b * io.H + p.h, nbh = (long long)io.B * io.H;
  if (PASS == kJoin)
    read_state(a.ws_s + (p.seg * nbh + bh) * sn);
  else if (PASS == kWhole && io.state && p.slot >= 0)
    read_state(io.state + ((long long)p.slot * io.H + p.h) * sn);

  TwoSum pending = {0.f, 0.f};  // sum of g that s does not have yet
  TwoSum all = {0.f, 0.f};      // and that of the segment

  if (p.t_lo < p.t_end) load_tile(0, p.t_lo);
  int st = 0;
  for (int t0 = p.t_lo; t0 < p.t_end; t0 += kStepTokens, st ^= 1) {
    copies_wait();
    __syncthreads();
    if (t0 + kStepTokens < p.t_end) load_tile(st ^ 1, t0 + kStepTokens);
    const int nt = min(kStepTokens, p.t_end - t0);
    const float* f;
    if constexpr (sizeof(T) == 4) {
      f = reinterpret_cast<const float*>(raw(st));
    } else {
      float* w = reinterpret_cast<float*>(smem + lay.off_f);
      const uint2* src = reinterpret_cast<const uint2*>(raw(st));
      for (int e = tid; e < nt * lay.row / 4; e += threads) {
        const uint2 v = src[e];
        reinterpret_cast<float4*>(w)[e] =
            make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                        __uint_as_float(v.y & 0xFFFF0000u));
      }
      __syncthreads();
      f = w;
    }
    // Lane t: g of token t and its sum from the tile's start.
    const float own = lane < nt ? raw_g(st)[lane] : 0.f;
    TwoSum sum = {own, 0.f};
#pragma unroll
    for (int m = 1; m < kStepTokens; m *= 2) {
      const TwoSum x = sum.from_lane(lane - m);
      if (lane >= m) sum = x + sum;
    }
    const bool lazy = __all_sync(0xFFFFFFFFu, fabsf(sum.hi) <= kLazy);  // not with a NaN either
    if (pending.hi != 0.f) {
      const float e = pending.exp(1.f);
      const uint64_t both = pack2(e, e);
#pragma unroll
      for (int i = 0; i < kRows / 2; ++i)
#pragma unroll
        for (int c = 0; c < kCols; ++c) s[i][c] = mul2(s[i][c], both);
    }
    const float up = lazy ? sum.exp(-1.f) : 1.f, down = lazy ? sum.exp(1.f) * io.scale : io.scale,
                each = at_most_finite(exp2_fast(kLog2e * own));
    pending = lazy ? sum.from_lane(nt - 1) : TwoSum{0.f, 0.f};
    if (PASS == kReduce) {
      if (lazy && fabsf(all.hi) <= 3.0e38f) {
        all = all + pending;
      } else {  // an infinite sum has no remainder
        for (int t = 0; t < nt; ++t) all.hi += __shfl_sync(0xFFFFFFFFu, own, t);
      }
    }

    for (int t = 0; t < nt; ++t, f += lay.row) {
      const float u = __shfl_sync(0xFFFFFFFFu, up, t);
      if (!lazy) {
        const float e = __shfl_sync(0xFFFFFFFFu, each, t);
        const uint64_t both = pack2(e, e);
#pragma unroll
        for (int i = 0; i < kRows / 2; ++i)
#pragma unroll
          for (int c = 0; c < kCols; ++c) s[i][c] = mul2(s[i][c], both);
      }
      const float4* kp = reinterpret_cast<const float4*>(f + DK) + r;
      const float4 v = *reinterpret_cast<const float4*>(f + 2 * DK + col);
      const uint64_t v2[kCols] = {pack2(v.x * u, v.x * u), pack2(v.y * u, v.y * u), pack2(v.z * u, v.z * u),
                                  pack2(v.w * u, v.w * u)};
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const float4 w = kp[i * R];
        const uint64_t k0 = pack2(w.x, w.y), k1 = pack2(w.z, w.w);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          s[2 * i][c] = fma2(k0, v2[c], s[2 * i][c]);
          s[2 * i + 1][c] = fma2(k1, v2[c], s[2 * i + 1][c]);
        }
      }
      if (PASS == kReduce) continue;
      uint64_t acc[kCols];
      const float4* qp = reinterpret_cast<const float4*>(f) + r;
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        const float4 w = qp[i * R];
        const uint64_t q0 = pack2(w.x, w.y), q1 = pack2(w.z, w.w);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          acc[c] = i == 0 ? mul2(q0, s[0][c]) : fma2(q0, s[2 * i][c], acc[c]);
          acc[c] = fma2(q1, s[2 * i + 1][c], acc[c]);
        }
      }
      float o[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float x, y;
        unpack2(acc[c], x, y);
        o[c] = x + y;
      }
      // Sums over the R lanes: in each step a lane hands half of its columns over and keeps the other half.
      int at = 0;
#pragma unroll
      for (int n = kCols / 2, m = R / 2; m > 0; m /= 2) {
        if (n > 0) {
          const bool upper = r & m;
#pragma unroll
          for (int c = 0; c < n; ++c) {
            const float give = upper ? o[c] : o[c + n], keep = upper ? o[c + n] : o[c];
            o[c] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, m);
          }
          at += upper ? n : 0;
          n /= 2;
        } else {
          o[0] += __shfl_xor_sync(0xFFFFFFFFu, o[0], m);
        }
      }
      constexpr int left = kCols / R < 1 ? 1 : kCols / R;
      const float dn = __shfl_sync(0xFFFFFFFFu, down, t);
#pragma unroll
      for (int c = 0; c < left; ++c) so[t * lay.vc + col + at + c] = o[c] * dn;
    }
    if (PASS != kReduce) {
      __syncthreads();
      if (a.vec_o) {
        const int NP = lay.vc / V;
        for (int e = tid; e < nt * NP; e += threads) {
          const int t = e / NP, c = e % NP * V;
          if (c >= nv) continue;
          float x[V];
#pragma unroll
          for (int j = 0; j < V; ++j) x[j] = so[t * lay.vc + c + j];
          *reinterpret_cast<uint4*>(go + (t0 + t) * ots + c) = Piece<T>::pack(x);
        }
      } else {
        for (int t = warp; t < nt; t += warps)
          for (int c = lane; c < nv; c += 32) from_f32(so[t * lay.vc + c], go + (t0 + t) * ots + c);
      }
    }
  }
  if (PASS != kReduce) {
    for (int t = max(p.t_end, p.t_lo); t < p.t_hi; ++t)  // no token here
      for (int c = tid; c < nv; c += threads) from_f32(0.f, go + t * ots + c);
  }
  const float end = pending.exp(1.f);
  if (PASS == kReduce) {
    write_state(a.ws_s + (p.seg * nbh + bh) * sn, end);
    if (p.vt == 0 && tid == 0) a.ws_g[p.seg * nbh + bh] = all.hi + all.lo;
  } else if (p.last && io.state_out && p.slot >= 0) {
    write_state(io.state_out + ((long long)p.slot * io.H + p.h) * sn, end);
  }
}

// The state in front of every segment, in the place of the segment's own end: h_0 = state, h_{j+1} = e^{G_j} h_j +
// end_j.  Eight segments' ends are asked for at a time.
__global__ void __launch_bounds__(256) front_kernel(const __grid_constant__ LinearArgs a) {
  wait_previous();
  allow_next();
  const sdm_linear_args& io = a.io;
  const long long sn = (long long)io.dk * io.dv, nbh = (long long)io.B * io.H;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  if (e >= sn * nbh) return;
  const long long bh = e / sn;
  const int b = int(bh / io.H), h = int(bh - (long long)b * io.H);
  const int slot = row_slot(io.slots, b, io.n_slots, nullptr);
  float x = io.state && slot >= 0 ? io.state[((long long)slot * io.H + h) * sn + (e - bh * sn)] : 0.f;
  const int n = a.segments - 1;
  for (int j0 = 0; j0 < n; j0 += 8) {
    float end[8], g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < n) {
        end[j] = a.ws_s[(j0 + j) * nbh * sn + e];
        g[j] = a.ws_g[(j0 + j) * nbh + bh];
      }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j0 + j < n) {
        a.ws_s[(j0 + j) * nbh * sn + e] = x;
        x = carried_up(x, g[j], kLog2e, end[j]);
      }
  }
  a.ws_s[n * nbh * sn + e] = x;
}

// ---- one token ----

constexpr int kTokenThreads = 128;
constexpr int kTokenCols = 32;  // state columns of a block

// A block takes 32 columns of a state: 128 consecutive bytes of each row, a float4 (V = 4) or a float a thread, rows dealt
// out in turn, eight under way.
template <typename T, int V>
__global__ void __launch_bounds__(kTokenThreads) token_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int CG = kTokenCols / V, RG = kTokenThreads / CG, kAhead = V == 4 ? 8 : 16;
  __shared__ float sq[SDM_MAX_LINEAR_D], sk[SDM_MAX_LINEAR_D];
  __shared__ float part[RG][kTokenCols];
  const sdm_linear_args& io = a.io;
  const int tid = threadIdx.x;
  unsigned id = blockIdx.x;
  const int vt = int(id % unsigned(a.vtiles));
  id /= unsigned(a.vtiles);
  const int h = int(id % unsigned(io.H)), b = int(id / unsigned(io.H)), hk = h / (io.H / io.Hk);
  const int asked = asked_slot(io.slots, b);
  const int dk = io.dk, dv = io.dv, c0 = vt * kTokenCols, cg = tid % CG, rg = tid / CG;
  const int c = c0 + cg * V;
  const T* q = static_cast<const T*>(io.q) + b * io.q_bs + (long long)hk * dk;
  const T* k = static_cast<const T*>(io.k) + b * io.k_bs + (long long)hk * dk;
  for (int i = tid; i < dk; i += kTokenThreads) sq[i] = to_f32(q[i]), sk[i] = to_f32(k[i]);
  float v[V];
  const T* pv = static_cast<const T*>(io.v) + b * io.v_bs + (long long)h * dv;
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = c + j < dv ? to_f32(pv[c + j]) : 0.f;
  const float e = io.g ? at_most_finite(expf(io.g[b * io.g_bs + h])) : 1.0f;
  const int length = row_length(io.lengths, b, 1);
  const int slot = checked_slot(io.slots, asked, io.n_slots, a.dev_err);
  __syncthreads();
  float o[V];
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = 0.f;
  const long long at = slot < 0 ? 0 : ((long long)slot * io.H + h) * dk * dv + c;
  const bool live = slot >= 0 && length > 0;
  if (slot >= 0 && c < dv) {
    const float* src = io.state ? io.state + at : nullptr;
    float* dst = io.state_out ? io.state_out + at : nullptr;
    for (int r0 = rg; r0 < dk; r0 += RG * kAhead) {
      float s[kAhead][V];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r0 + i * RG;
#pragma unroll
        for (int j = 0; j < V; ++j) s[i][j] = 0.f;
        if (row < dk && src) {
          const float* f = src + (long long)row * dv;
          if constexpr (V == 4) {
            const float4 w = __ldcs(reinterpret_cast<const float4*>(f));
            s[i][0] = w.x, s[i][1] = w.y, s[i][2] = w.z, s[i][3] = w.w;
          } else {
            s[i][0] = __ldcs(f);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r0 + i * RG;
        if (row >= dk) break;
        if (live) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            s[i][j] = fmaf(e, s[i][j], sk[row] * v[j]);
            o[j] = fmaf(sq[row], s[i][j], o[j]);
          }
        }
        if (dst) {
          float* f = dst + (long long)row * dv;
          if constexpr (V == 4)
            __stcs(reinterpret_cast<float4*>(f), make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
          else
            __stcs(f, s[i][0]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) part[rg][cg * V + j] = o[j];
  __syncthreads();
  if (tid < kTokenCols && c0 + tid < dv) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < RG; ++i) sum += part[i][tid];
    from_f32(live ? sum * io.scale : 0.f, static_cast<T*>(io.o) + ((long long)b * io.H + h) * dv + c0 + tid);
  }
}

template <typename T>
int launch_token(LinearArgs& a, cudaStream_t s) {
  a.vtiles = (a.io.dv + kTokenCols - 1) / kTokenCols;
  const long long blocks = (long long)a.io.B * a.io.H * a.vtiles;
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  if (a.vec_s)
    token_kernel<T, 4><<<unsigned(blocks), kTokenThreads, 0, s>>>(a);
  else
    token_kernel<T, 1><<<unsigned(blocks), kTokenThreads, 0, s>>>(a);
  return last_launch_status();
}

template <typename T, int DK, int PASS>
int launch_pass(LinearArgs a, int warps, cudaStream_t s) {
  auto fn = step_kernel<T, DK, PASS>;
  const StepTile<T, DK> lay(warps);
  static PerDevice ready;
  if (ready.get([&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, StepTile<T, DK>(kStepWarps).bytes) ==
                       cudaSuccess ? 1 : -1;
      }) < 0)
    return SDM_ECUDA;
  a.vtiles = (a.io.dv + lay.vc - 1) / lay.vc;
  const long long blocks =
      (long long)a.vtiles * a.io.H * a.io.B * (PASS == kReduce ? a.segments - 1 : a.segments);
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(unsigned(warps * 32));
  cfg.dynamicSmemBytes = size_t(lay.bytes);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = PASS == kJoin ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, fn, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

template <typename T, int DK>
int launch_steps(const LinearArgs& a, cudaStream_t s) {
  const int need = (a.io.dv + Warp<DK>::cols - 1) / Warp<DK>::cols, warps = need < kStepWarps ? need : kStepWarps;
  if (a.segments <= 1) return launch_pass<T, DK, kWhole>(a, warps, s);
  int st = launch_pass<T, DK, kReduce>(a, warps, s);
  if (st == SDM_OK) st = launch_front(a, s);
  return st == SDM_OK ? launch_pass<T, DK, kJoin>(a, warps, s) : st;
}

template <typename T>
int launch_type(const LinearArgs& a, cudaStream_t s) {
  if (a.io.dk <= 32) return launch_steps<T, 32>(a, s);
  if (a.io.dk <= 64) return launch_steps<T, 64>(a, s);
  if (a.io.dk <= 128) return launch_steps<T, 128>(a, s);
  return launch_steps<T, 256>(a, s);
}

bool sizes_ok(int dtype, int B, int T, int H, int dk, int dv) {
  return !bad_dtype(dtype) && B >= 1 && T >= 0 && H >= 1 && dk >= 1 && dv >= 1;
}

// How a sequence is cut for step_kernel: a warp's piece of a state is a unit of work, and the card runs 16 of them an
// SM; twice the work pays from some three segments on (4 heads of 64 x 64 in fp32: 95 tokens whole 31 us, 96 in
// three segments 28; 2048 tokens of 100 heads of 128 x 128 in three 607, 128 heads whole 668).
void cut_steps(int B, int T, int H, int dk, int dv, int* segments, int* segment) {
  const int DK = dk <= 32 ? 32 : dk <= 64 ? 64 : dk <= 128 ? 128 : 256, cols = 32 / (DK / kRows) * kCols;
  const long long units = (long long)B * H * ((dv + cols - 1) / cols);
  long long n = 152 * 16 / units;
  n = n < T / (2 * kStepTokens) ? n : T / (2 * kStepTokens);
  if (n < 3) n = 1;
  const long long per = ((T + n - 1) / n + kStepTokens - 1) / kStepTokens * kStepTokens;
  *segment = n > 1 ? int(per) : T;
  *segments = n > 1 ? int((T + per - 1) / per) : 1;
}

// What of the output, the new states and the workspace overlaps anything else of the call.
bool overlap(const sdm_linear_args& io, const void* workspace, size_t workspace_bytes) {
  const long long es = io.dtype == SDM_F32 ? 4 : 2, qk = (long long)io.Hk * io.dk * es, vr = (long long)io.H * io.dv * es;
  const long long sn = 4LL * io.n_slots * io.H * io.dk * io.dv, on = (long long)io.B * io.T * vr, wn = (long long)workspace_bytes;
  auto rows = [&](const void* p, long long bs, long long ts, long long bytes, long long size) {
    return Extent{p, io.B, bs * size, io.T, ts * size, bytes};
  };
  const Extent state = dense(io.state, sn);
  for (const Extent& e : {rows(io.q, io.q_bs, io.q_ts, qk, es), rows(io.k, io.k_bs, io.k_ts, qk, es),
                          rows(io.v, io.v_bs, io.v_ts, vr, es), rows(io.g, io.g_bs, io.g_ts, 4LL * io.H, 4),
                          dense(io.lengths, 4LL * io.B), dense(io.slots, 4LL * io.B),
                          io.state == io.state_out ? Extent{} : state})
    if (meets(e, io.o, on) || meets(e, io.state_out, sn) || meets(e, workspace, wn)) return true;
  return meets(state, io.o, on) || meets(state, workspace, wn) || meets(dense(io.o, on), io.state_out, sn) ||
         meets(dense(io.o, on), workspace, wn) || meets(dense(io.state_out, sn), workspace, wn);
}

}  // namespace

int launch_front(const LinearArgs& a, cudaStream_t s) {
  const long long n = (long long)a.io.B * a.io.H * a.io.dk * a.io.dv, blocks = (n + 255) / 256;
  if (blocks > 0x7FFFFFFFLL) return SDM_EUNSUPPORTED;
  cudaLaunchAttribute attr[1] = {after_previous()};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, front_kernel, a) != cudaSuccess) return SDM_ECUDA;
  return last_launch_status();
}

}  // namespace sdm

using namespace sdm;

// What of the workspace a call with these sizes may need: the segments' states and sums of g, then copies of rows that
// are not multiples of 16 bytes.  Which form is taken, strides and addresses decide too.
namespace {

// From 32 tokens on chunks pay: 1024 heads of 128 x 128 take 66 us for 31 tokens one by one and 51 for 32 as a chunk,
// 128 heads 16 and 12.  Small heads that fill the card several times want 64: 1024 heads of 64 x 64 take 25 us for 31
// tokens one by one, 47 as a chunk.
bool tile_sizes(int dtype, int B, int T, int H, int dk, int dv) {
  const int least = dk * dv <= 64 * 64 && (long long)B * H > 4 * 152 ? 64 : 32;
  return dtype == SDM_BF16 && T >= least && dk <= SDM_LINEAR_TILE_D;
}
struct LinearSpace {
  size_t states = 0, pad = 0;
  LinearSpace(int dtype, int B, int T, int H, int Hk, int dk, int dv) {
    int segments, segment;
    cut_steps(B, T, H, dk, dv, &segments, &segment);
    if (tile_sizes(dtype, B, T, H, dk, dv)) {
      int n;
      cut_tiles(B, T, H, dv, &n, &segment);
      segments = n > segments ? n : segments;
      if (dk % 8 || dv % 8) pad = padded_bytes(B, T, H, Hk, dk, dv);
    }
    if (segments > 1) states = (size_t(segments) * B * H * (size_t(dk) * dv + 1 + tile_columns(dv)) * 4 + 255) / 256 * 256;
  }
};
}  // namespace

extern "C" size_t sdm_linear_attention_workspace_size(int dtype, int B, int T, int H, int Hk, int dk, int dv) {
  if (!sizes_ok(dtype, B, T, H, dk, dv) || Hk < 1 || H % Hk || dk > SDM_MAX_LINEAR_D || dv > SDM_MAX_LINEAR_D || T <= 1)
    return 0;
  const LinearSpace space(dtype, B, T, H, Hk, dk, dv);
  return space.states + space.pad;
}

static int linear_attention(const sdm_linear_args* args, void* workspace, size_t workspace_bytes, int* dev_err, void* stream,
                            const LinearStall* stall) {
  if (!args) return SDM_EINVAL;
  const sdm_linear_args& io = *args;
  if (!sizes_ok(io.dtype, io.B, io.T, io.H, io.dk, io.dv) || io.Hk < 1 || io.H % io.Hk) return SDM_EINVAL;
  if (io.dk > SDM_MAX_LINEAR_D || io.dv > SDM_MAX_LINEAR_D || (long long)io.B * io.T > 0x7FFFFFFFLL ||
      io.T > 0x7FFFFFFF - 1024 || (long long)io.B * io.H > 0x7FFFFFFLL)
    return SDM_EUNSUPPORTED;
  if ((io.state || io.state_out || io.slots) && io.n_slots < (io.slots ? 1 : io.B)) return SDM_EINVAL;
  const uintptr_t odd = io.dtype == SDM_F32 ? 3 : 1;
  auto off = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (off(io.state, 3) || off(io.state_out, 3) || off(io.g, 3) || off(io.lengths, 3) || off(io.slots, 3) ||
      off(dev_err, 3))
    return SDM_EALIGN;
  if (io.T > 0 && (!io.q || !io.k || !io.v || !io.o || off(io.q, odd) || off(io.k, odd) || off(io.v, odd) || off(io.o, odd)))
    return SDM_EALIGN;
  if (io.T == 0 && (io.state == io.state_out || !io.state_out)) return SDM_OK;

  LinearArgs a = {};
  a.io = io;
  a.dev_err = dev_err;
  if (stall) a.stall = *stall;
  cudaStream_t s = as_stream(stream);
  a.vec_s = io.dv % 4 == 0 && !off(io.state, 15) && !off(io.state_out, 15);
  if (io.T == 1) {
    if (stall) return SDM_EUNSUPPORTED;
    if (overlap(io, nullptr, 0)) return SDM_EOVERLAP;
    return io.dtype == SDM_F32 ? launch_token<float>(a, s) : launch_token<__nv_bfloat16>(a, s);
  }
  const int V = io.dtype == SDM_F32 ? 4 : 8;
  auto rows16 = [&](const void* p, long long bs, long long ts) { return !off(p, 15) && bs % V == 0 && ts % V == 0; };
  a.vec_qk = io.dk % V == 0 && rows16(io.q, io.q_bs, io.q_ts) && rows16(io.k, io.k_bs, io.k_ts);
  a.vec_v = io.dv % V == 0 && rows16(io.v, io.v_bs, io.v_ts);
  a.vec_o = io.dv % V == 0 && !off(io.o, 15);
  auto steps_on = [&](long long bs, long long ts) { return ts > 0 && (io.B == 1 || bs > 0); };
  const LinearSpace space(io.dtype, io.B, io.T, io.H, io.Hk, io.dk, io.dv);
  const size_t need = space.states + space.pad;
  const bool rows_fit = a.vec_qk && a.vec_v && a.vec_o && steps_on(io.q_bs, io.q_ts) && steps_on(io.k_bs, io.k_ts) &&
                        steps_on(io.v_bs, io.v_ts);
  const bool tiles = tile_sizes(io.dtype, io.B, io.T, io.H, io.dk, io.dv) && (rows_fit || space.pad);
  if (stall && !tiles) return SDM_EUNSUPPORTED;
  if (tiles)
    cut_tiles(io.B, io.T, io.H, io.dv, &a.segments, &a.segment);
  else
    cut_steps(io.B, io.T, io.H, io.dk, io.dv, &a.segments, &a.segment);
  if (need) {
    if (!aligned16(workspace)) return SDM_EALIGN;
    if (workspace_bytes < need) return SDM_ENOSPACE;
    a.ws_s = static_cast<float*>(workspace);
    a.ws_g = a.ws_s + size_t(a.segments) * io.B * io.H * io.dk * io.dv;
    a.ws_stop = reinterpret_cast<int*>(a.ws_g + size_t(a.segments) * io.B * io.H);
  }
  if (overlap(io, need ? workspace : nullptr, need)) return SDM_EOVERLAP;
  if (tiles) return launch_tiles(a, rows_fit ? nullptr : static_cast<uint8_t*>(workspace) + space.states, s);
  return io.dtype == SDM_F32 ? launch_type<float>(a, s) : launch_type<__nv_bfloat16>(a, s);
}

extern "C" int sdm_linear_attention(const sdm_linear_args* args, void* workspace, size_t workspace_bytes, int* dev_err,
                                    void* stream) {
  return linear_attention(args, workspace, workspace_bytes, dev_err, stream, nullptr);
}

extern "C" int sdm_test_linear_stall(const sdm_linear_args* args, void* workspace, size_t workspace_bytes, int pass, int block,
                                     int chunk, int load, unsigned long long wait_ns, int* dev_err, void* stream) {
  if (pass < kWhole || pass > kJoin || block < 0 || chunk < 0 || load < 0 || load > 2 || wait_ns < 100000ull ||
      wait_ns > 1000000000ull || !dev_err)
    return SDM_EINVAL;
  LinearStall stall;
  stall.pass = pass, stall.block = block, stall.chunk = chunk, stall.load = load, stall.wait_ns = wait_ns;
  return linear_attention(args, workspace, workspace_bytes, dev_err, stream, &stall);
}
