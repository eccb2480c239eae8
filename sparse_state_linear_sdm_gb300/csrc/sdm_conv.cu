// Short causal depthwise convolution in front of a recurrent layer, over prompts and for single
// tokens.
//
//   y[b,t,d] = act(bias[d] + sum_{j<K} w[d,j] u[b, t-K+1+j, d])
//
// where u is the K-1 inputs carried from before token 0 (the state) followed by x, and the new
// state is the last K-1 inputs of each sequence.  2K flop for each element read and written
// once: HBM bounds it, so each thread keeps its 16-byte piece of channels (8 bf16 or 4 fp32)
// and walks a strip of tokens with the last K-1 inputs beside it: every input is read once,
// except the K-1 tokens before a strip.  The next kAhead tokens are always under way, as raw words,
// and two multiply-adds go in one instruction: 8 x 4096 x 4096 bf16 with silu and four taps takes
// 99 us, 5.4 TB/s (0.80 of a copy's rate); with four tokens under way 110 us, with weights loaded one
// by one and inputs held as fp32 266 us.  fp32 takes 169 us (0.94), 185 with eight taps.
//
// The window and the weights are in registers for up to four taps in bf16 and for any number in fp32.
// The bound of 128 registers was chosen at four taps (105 us without it); more taps of 8 channels do
// not fit in it and spill (1.4 KB a thread at eight): 156, 210, 251 and 361 us with 5 to 8 taps,
// where HBM would let them take 79.
//
// A token is a strip of one, whose thread still goes through the arithmetic of kAhead tokens: 10 us for
// 256 x 4096 with four taps, 19 for rows off 16 bytes (an element a thread), 37 with eight taps.
#include "sdm_layers.cuh"

namespace sdm {
namespace {

constexpr int kConvThreads = 64;
constexpr int kAhead = 8;  // tokens under way: a register word each, reloaded as soon as it is taken
constexpr int kMinStrip = 8;  // shortest strip: longer than the window
static_assert(kMinStrip == SDM_CONV_IN_PLACE, "so many tokens are one strip");

struct ConvArgs {
  const void* x;
  long long x_bs, x_ts;  // elements between sequences and between tokens
  const void* w;
  const void* bias;
  int w_dt, B, T, D, act;
  const void* state;
  void* state_out;
  int n_slots;
  const int32_t* lengths;
  const int32_t* slots;
  void* y;
  int* dev_err;
  int strip, strips, pieces;  // tokens a thread, strips a sequence, pieces a row
  bool w_vec;                 // w and bias start on 8 bytes
};

// N weights from element i on; 8 bytes at a time where `vec` says that they start there.
template <int N, int V>
__device__ __forceinline__ void load_weights(const void* p, int dt, size_t i, bool vec, float (&w)[N]) {
  if (V > 1 && vec) {
    if (dt == SDM_F32) {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const float2 v = reinterpret_cast<const float2*>(static_cast<const float*>(p) + i)[k];
        w[2 * k] = v.x, w[2 * k + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
        const uint2 v = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i)[k];
        w[4 * k] = __uint_as_float(v.x << 16), w[4 * k + 1] = __uint_as_float(v.x & 0xFFFF0000u);
        w[4 * k + 2] = __uint_as_float(v.y << 16), w[4 * k + 3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      w[k] = dt == SDM_F32 ? static_cast<const float*>(p)[i + k]
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i + k]);
  }
}

// V channels: as they lie in memory (one 16-byte word where V is a whole piece, else one element),
// and as numbers (pairs, for two operations an instruction, or one).
template <typename T, int V>
struct Channels {
  static constexpr int n = V / 2;
  using word = uint4;
  using num = uint64_t;
  __device__ static word zero() { return make_uint4(0, 0, 0, 0); }
  __device__ static void load(const word& w, num (&v)[n]) {
    float f[V];
    Piece<T>::load(w, f);
    join(f, v);
  }
  __device__ static void join(const float (&f)[V], num (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
  __device__ static num fma(num a, num b, num c) { return fma2(a, b, c); }
  __device__ static num act(num v) {
    float a, b;
    unpack2(v, a, b);
    return mul2(v, pack2(sigmoid(a), sigmoid(b)));
  }
  __device__ static word pack(const num (&v)[n]) {
    float f[V];
#pragma unroll
    for (int i = 0; i < n; ++i) unpack2(v[i], f[2 * i], f[2 * i + 1]);
    return Piece<T>::pack(f);
  }
};
template <typename T>
struct Channels<T, 1> {
  static constexpr int n = 1;
  using word = T;
  using num = float;
  __device__ static word zero() { return T(0.f); }
  __device__ static void load(const word& w, num (&v)[1]) { v[0] = to_f32(w); }
  __device__ static void join(const float (&f)[1], num (&v)[1]) { v[0] = f[0]; }
  __device__ static num fma(num a, num b, num c) { return fmaf(a, b, c); }
  __device__ static num act(num v) { return silu(v); }
  __device__ static word pack(const num (&v)[1]) {
    T r;
    from_f32(v[0], &r);
    return r;
  }
};

template <typename T, int K, int V, bool ACT>
__global__ void __launch_bounds__(kConvThreads, 8) conv_kernel(const __grid_constant__ ConvArgs a) {
  using C = Channels<T, V>;
  using word = typename C::word;
  using num = typename C::num;
  const unsigned id = blockIdx.x * kConvThreads + threadIdx.x;  // under 2^32, see the launch
  const unsigned row = id / unsigned(a.pieces);
  const int piece = int(id - row * unsigned(a.pieces));
  const int b = int(row / unsigned(a.strips)), strip = int(row - unsigned(b) * unsigned(a.strips));
  if (b >= a.B) return;
  const int d = piece * V;
  const int asked = asked_slot(a.slots, b);
  const int given = row_length(a.lengths, b, a.T);
  const int t0 = strip * a.strip, t1 = min(t0 + a.strip, a.T);
  const T* x = static_cast<const T*>(a.x) + b * a.x_bs + d;
  auto token = [&](int t) {  // zero past the sequence
    return t < given ? *reinterpret_cast<const word*>(x + t * a.x_ts) : C::zero();
  };

  word next[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) next[k] = t0 + k < t1 ? token(t0 + k) : C::zero();

  num w[K][C::n], bias[C::n];
  {
    float f[K * V], tap[V];
    load_weights<K * V, V>(a.w, a.w_dt, size_t(d) * K, a.w_vec, f);  // channel i, tap j at i * K + j
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) tap[i] = f[i * K + j];
      C::join(tap, w[j]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) tap[i] = 0.f;
    if (a.bias) load_weights<V, V>(a.bias, a.w_dt, d, a.w_vec, tap);
    C::join(tap, bias);
  }

  const int slot = checked_slot(a.slots, asked, a.n_slots, a.dev_err);
  const int len = slot < 0 ? 0 : given;
  const int end = min(t1, len);  // tokens of this strip that exist: [t0, end)
  const size_t srow = size_t(max(slot, 0)) * (K - 1) * a.D + d;
  num win[K - 1][C::n];
  {
    word old[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      if (t0 > 0)
        old[j] = token(t0 - (K - 1) + j);
      else
        old[j] = a.state && slot >= 0
                     ? *reinterpret_cast<const word*>(static_cast<const T*>(a.state) + srow + size_t(j) * a.D)
                     : C::zero();
      C::load(old[j], win[j]);
    }
    if (t0 == 0 && slot >= 0 && a.state_out) {
      // This thread alone reads its channels' old state (above) and writes the new one, so the
      // state may be updated in place.
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int t = len - (K - 1) + j;
        word v = C::zero();
        if (t >= 0) {
          v = token(t);
        } else {  // a sequence shorter than the window keeps the end of the old state
#pragma unroll
          for (int o = 0; o < K - 1; ++o)
            if (o == t + K - 1) v = old[o];
        }
        *reinterpret_cast<word*>(static_cast<T*>(a.state_out) + srow + size_t(j) * a.D) = v;
      }
    }
  }

  T* y = static_cast<T*>(a.y) + (size_t(b) * a.T + t0) * a.D + d;
  const T* ahead = x + (t0 + kAhead) * a.x_ts;
  int t = t0;
  for (; t < end; t += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      num in[C::n], o[C::n];
      C::load(next[k], in);
      if (t + kAhead + k < end) next[k] = *reinterpret_cast<const word*>(ahead);
      ahead += a.x_ts;
#pragma unroll
      for (int i = 0; i < C::n; ++i) {
        num s = bias[i];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) s = C::fma(w[j][i], win[j][i], s);
        s = C::fma(w[K - 1][i], in[i], s);
        o[i] = ACT ? C::act(s) : s;
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) win[j][i] = win[j + 1][i];
        win[K - 2][i] = in[i];
      }
      if (t + k < end) *reinterpret_cast<word*>(y) = C::pack(o);
      y += a.D;
    }
  }
  for (t = max(t0, end); t < t1; ++t)
    *reinterpret_cast<word*>(static_cast<T*>(a.y) + (size_t(b) * a.T + t) * a.D + d) = C::zero();
}

template <typename T, int K, int V>
void launch_act(const ConvArgs& a, unsigned blocks, cudaStream_t s) {
  if (a.act == SDM_ACT_SILU)
    conv_kernel<T, K, V, true><<<blocks, kConvThreads, 0, s>>>(a);
  else
    conv_kernel<T, K, V, false><<<blocks, kConvThreads, 0, s>>>(a);
}

template <typename T, int K>
int launch_k(const ConvArgs& a, bool vec, cudaStream_t s) {
  const long long blocks =
      ((long long)a.B * a.strips * a.pieces + kConvThreads - 1) / kConvThreads;
  if (blocks * kConvThreads > 0xFFFFFFFFLL) return SDM_EUNSUPPORTED;
  if (vec)
    launch_act<T, K, Piece<T>::n>(a, unsigned(blocks), s);
  else
    launch_act<T, K, 1>(a, unsigned(blocks), s);
  return last_launch_status();
}

template <typename T>
int launch_t(const ConvArgs& a, int K, bool vec, cudaStream_t s) {
  switch (K) {
    case 2: return launch_k<T, 2>(a, vec, s);
    case 3: return launch_k<T, 3>(a, vec, s);
    case 4: return launch_k<T, 4>(a, vec, s);
    case 5: return launch_k<T, 5>(a, vec, s);
    case 6: return launch_k<T, 6>(a, vec, s);
    case 7: return launch_k<T, 7>(a, vec, s);
    case 8: return launch_k<T, 8>(a, vec, s);
    default: return SDM_EUNSUPPORTED;
  }
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" int sdm_causal_conv(const void* x, long long x_bstride, long long x_tstride, int dt,
                               const void* w, const void* bias, int w_dt, int B, int T, int D,
                               int K, int act, const void* state, void* state_out, int n_slots,
                               const int32_t* lengths, const int32_t* slots, void* y,
                               int* dev_err, void* stream) {
  if (B < 1 || T < 0 || D < 1 || K < 2 || bad_dtype(dt) || bad_dtype(w_dt)) return SDM_EINVAL;
  if (act != SDM_ACT_NONE && act != SDM_ACT_SILU) return SDM_EINVAL;
  // A token's index may run past T by a strip and the tokens under way, and stays an int.
  constexpr int kPast = 256;
  if (K > SDM_MAX_CONV || (long long)B * T > 0x7FFFFFFFLL || T > 0x7FFFFFFF - kPast || D > 0x7FFFFFF)
    return SDM_EUNSUPPORTED;
  if ((state || state_out || slots) && n_slots < (slots ? 1 : B)) return SDM_EINVAL;
  const int es = dt == SDM_F32 ? 4 : 2;
  const uintptr_t odd = uintptr_t(es - 1), wodd = uintptr_t(w_dt == SDM_F32 ? 3 : 1);
  auto off = [](const void* p, uintptr_t m) { return (reinterpret_cast<uintptr_t>(p) & m) != 0; };
  if (!w || off(w, wodd) || off(bias, wodd) || off(state, odd) || off(state_out, odd) ||
      off(lengths, 3) || off(slots, 3) || off(dev_err, 3))
    return SDM_EALIGN;
  if (T > 0 && (!x || !y || off(x, odd) || off(y, odd))) return SDM_EALIGN;
  if (T == 0 && (state == state_out || !state_out)) return SDM_OK;
  const long long row = (long long)D * es, wes = w_dt == SDM_F32 ? 4 : 2, taps = K - 1;
  const Extent ex{x, B, x_bstride * es, T, x_tstride * es, row};
  const long long yn = (long long)B * T * row;
  // y as x: every strip but the first reads the end of the one before it, which another thread may
  // have overwritten; so may the first, which keeps the sequence's end as the state.
  const bool in_place = x == y && T <= kMinStrip && (B == 1 || x_bstride == (long long)T * D) &&
                        (T == 1 || x_tstride == D);
  for (const Extent& e : {in_place ? Extent{} : ex, dense(w, wes * D * K), dense(bias, wes * D),
                          dense(state, n_slots * taps * row), dense(state_out, n_slots * taps * row),
                          dense(lengths, 4LL * B), dense(slots, 4LL * B)})
    if (meets(e, y, yn)) return SDM_EOVERLAP;
  const long long sn = n_slots * taps * row;
  for (const Extent& e : {ex, dense(w, wes * D * K), dense(bias, wes * D),
                          state == state_out ? Extent{} : dense(state, sn), dense(lengths, 4LL * B),
                          dense(slots, 4LL * B)})
    if (meets(e, state_out, sn)) return SDM_EOVERLAP;

  const int V = 16 / es;
  // 16-byte pieces where every row of every operand starts on 16 bytes, else single elements.
  const bool vec = D % V == 0 && x_bstride % V == 0 && x_tstride % V == 0 && !off(x, 15) &&
                   !off(y, 15) && !off(state, 15) && !off(state_out, 15);
  ConvArgs a{x,     x_bstride, x_tstride, w,     bias, w_dt,    B, T, D,
             act,   state,     state_out, n_slots, lengths, slots, y, dev_err, 0, 0, 0, false};
  a.pieces = vec ? D / V : D;
  a.w_vec = !off(w, 7) && !off(bias, 7);
  // Strips of 128 tokens (the K-1 tokens read twice and the weights are then a small part),
  // shorter ones where that leaves the card's threads short.
  a.strip = 128;
  while (a.strip > kMinStrip &&
         (long long)B * ((T + a.strip - 1) / a.strip) * a.pieces < 152LL * 1024)
    a.strip /= 2;
  a.strips = T > 0 ? (T + a.strip - 1) / a.strip : 1;
  return dt == SDM_F32 ? launch_t<float>(a, K, vec, as_stream(stream))
                       : launch_t<__nv_bfloat16>(a, K, vec, as_stream(stream));
}
