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
//
// 16,384 x 16 groups of 128 with a gate: 61 us, 0.81 of the HBM floor; the stream alone, 16,384 x 2048, 55 (0.72).  Rows
// off 16 bytes are read element by element: everything of 4099 x 1537, bf16 with an fp32 stream, takes 41 (0.50).
// Beyond 4096 channels the sums live in shared memory (4096 x 8192 with everything 174 us, 282 in registers that spilled).
#pragma once

#include <type_traits>

#include "sdm_norm.cuh"

namespace sdm {

struct NormBackward {
  sdm_norm_args io;
  const void *r, *dy, *dr;
  long long r_rs, dy_rs, dr_rs;
  void *dx, *dres, *dgate;
  void *dafter, *dscale, *dweight;
  float* part;  // [slots][kinds][D]
  int slots;    // teams of a group
  int kinds;    // sums wanted
};

// What a call has of the gradient: bits, known where an instance is compiled.  Decided at run time, every one of them costs
// branches and registers: 32,768 x 1000 with all of them takes 169 us so and 97 as its own instance, the norm and gate over
// heads 82 and 61, the stream alone 68 and 55.  The sets below have an instance; the rest share kAny, among them the stream
// with a scale or a gate and no inner norm.
enum NormParts { kStream = 1, kAfter = 2, kGate = 4, kScale = 8, kAny = 16 };  // kGate: silu
constexpr bool norm_has(int kind, int part) { return kind == kAny || (kind & part); }
constexpr bool norm_small(int kind) { return kind == kStream || kind == kAfter || kind == (kAfter | kGate); }
constexpr int sm_threads(int kind, int pieces) { return pieces > 1 || !norm_small(kind) ? 512 : 768; }  // of an SM, by registers

// f(kind) of the instance for a set of parts.
template <typename F>
auto norm_instance(int parts, F f) {
  switch (parts) {
    case kStream: return f(std::integral_constant<int, kStream>());
    case kAfter: return f(std::integral_constant<int, kAfter>());
    case kAfter | kGate: return f(std::integral_constant<int, kAfter | kGate>());
    case kStream | kAfter: return f(std::integral_constant<int, kStream | kAfter>());
    case kStream | kAfter | kScale: return f(std::integral_constant<int, kStream | kAfter | kScale>());
    case kStream | kAfter | kGate | kScale: return f(std::integral_constant<int, kStream | kAfter | kGate | kScale>());
    default: return f(std::integral_constant<int, kAny>());
  }
}

template <typename TX, typename TR>
int launch_norm_backward(const NormBackward& a, int parts, bool vec, cudaStream_t s);

namespace {

// Sums over rows of a thread's channels: in registers, or, where there are too many of them, in dynamic shared memory.
template <int E, int BLOCK, bool SHARED>
struct Sum {
  float v[SHARED ? 1 : E];
  float4* s;
  __device__ explicit Sum(float4* at) : s(at + threadIdx.x) {
    if constexpr (SHARED) {
#pragma unroll
      for (int k = 0; k < E / 4; ++k) s[k * BLOCK] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
    }
  }
  // += a b, by element
  __device__ void add(const float (&a)[E], const float (&b)[E]) {
    if constexpr (SHARED) {
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        float4 x = s[k * BLOCK];
        x.x = fmaf(a[4 * k], b[4 * k], x.x), x.y = fmaf(a[4 * k + 1], b[4 * k + 1], x.y);
        x.z = fmaf(a[4 * k + 2], b[4 * k + 2], x.z), x.w = fmaf(a[4 * k + 3], b[4 * k + 3], x.w);
        s[k * BLOCK] = x;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = fmaf(a[e], b[e], v[e]);
    }
  }
  __device__ void get(float (&o)[E]) const {
    if constexpr (SHARED) {
#pragma unroll
      for (int k = 0; k < E / 4; ++k) {
        const float4 x = s[k * BLOCK];
        o[4 * k] = x.x, o[4 * k + 1] = x.y, o[4 * k + 2] = x.z, o[4 * k + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = v[e];
    }
  }
};
constexpr bool shared_sums(int kind, int pieces) { return !norm_small(kind) && pieces > 1; }
constexpr int shared_sums_bytes(int kind, int pieces, int block) {
  return shared_sums(kind, pieces) ? 3 * 8 * pieces * 4 * block : 0;
}

template <typename TX, typename TR, int TPR, int P, bool VEC, int KIND>
__global__ void __launch_bounds__(norm_block(TPR), sm_threads(KIND, P) / norm_block(TPR))
    backward_kernel(const __grid_constant__ NormBackward a) {
  // kAny's long rows have no registers left to ask for more at a time (4099 x 1537: 55 us, 64 if they do).
  typedef Row<TPR, P, VEC, KIND != kAny || TPR <= 32> R;
  constexpr int E = R::E, RPB = norm_block(TPR) / TPR, W = norm_block(TPR) / 32;
  constexpr int A = norm_has(KIND, kAfter), S = norm_has(KIND, kStream), K = 2 * S + A;  // sums of the first round
  constexpr int kWeights = A + S + norm_has(KIND, kScale);
  __shared__ float part1[2][W][K], part2[2][W][1];
  __shared__ Kept<R, norm_block(TPR), kWeights> kept;
  const sdm_norm_args& io = a.io;
  const int t = threadIdx.x % TPR, n = io.D / io.groups;
  const unsigned team = blockIdx.x * RPB + threadIdx.x / TPR;
  const unsigned slot = team / unsigned(io.groups), group = team % unsigned(io.groups);
  const bool used = slot < unsigned(a.slots);
  const long long off = (long long)group * n;
  const float rn = 1.0f / float(n);
  auto has = [](int part, bool asked) { return KIND == kAny ? asked : (KIND & part) != 0; };
  const bool weight = has(kStream, a.dy), after = has(kAfter, io.after), gate = has(kGate, io.gate),
             scale = has(kScale, io.scale), silu_gate = KIND != kAny || io.act == SDM_ACT_SILU;
  const bool from_r = !weight || a.dr;  // dr comes in
  allow_next();

  extern __shared__ float4 sums_at[];
  typedef Sum<E, norm_block(TPR), shared_sums(KIND, P)> Sums;
  Sums sum_after(sums_at), sum_scale(sums_at + E / 4 * norm_block(TPR)), sum_weight(sums_at + E / 2 * norm_block(TPR));

  // A row as it lies in memory; the next one is asked for while this one is worked on.
  typename R::template Raw<TX> rx, rz, rdy;
  typename R::template Raw<TR> rr, rdr;
  const TX* px = static_cast<const TX*>(io.x) + (after || gate || scale ? slot * io.x_rs + off : 0);
  const TX* pz = static_cast<const TX*>(io.gate) + (gate ? slot * io.gate_rs + off : 0);
  const TX* pdy = static_cast<const TX*>(a.dy) + (weight ? slot * a.dy_rs + off : 0);
  const TR* pr = static_cast<const TR*>(a.r) + (weight ? slot * a.r_rs + off : 0);
  const TR* pdr = static_cast<const TR*>(a.dr) + (from_r ? slot * a.dr_rs + off : 0);
  const long long out = slot * (long long)io.D + off, step = a.slots * (long long)io.D;
  TX* dx = static_cast<TX*>(a.dx) + (a.dx ? out : 0);
  TX* dgate = static_cast<TX*>(a.dgate) + (a.dgate ? out : 0);
  TR* dres = static_cast<TR*>(a.dres) + (a.dres ? out : 0);
  auto ask = [&](long long m0) {
    if (R::kAlone && m0 + slot >= io.M) return;
    const int cols = R::kAlone || (used && m0 + slot < io.M) ? n : 0;
    if (after || gate || scale) rx.ask(px, t, cols), px += a.slots * io.x_rs;
    if (gate) rz.ask(pz, t, cols), pz += a.slots * io.gate_rs;
    if (weight) {
      rdy.ask(pdy, t, cols), pdy += a.slots * a.dy_rs;
      rr.ask(pr, t, cols), pr += a.slots * a.r_rs;
    }
    if (from_r) rdr.ask(pdr, t, cols), pdr += a.slots * a.dr_rs;
  };
  constexpr bool kAhead = P == 1 || (P == 2 && norm_small(KIND));  // otherwise it takes more registers than it gains
  if (kAhead) ask(0);
  const long long at = used ? off : 0;
  const int mine = used ? n : 0;
  auto keep = [&](int which, const void* p) { kept.put(which, p, io.w_dtype, at, t, mine); };
  auto weights = [&](int which, const void* p, float (&w)[E]) { kept.get(which, p, io.w_dtype, at, t, mine, w); };
  if (after) keep(0, io.after);
  if (weight) keep(A, io.weight);
  if (scale) keep(A + S, io.scale);

  int turn = 0;
  for (long long m0 = 0; m0 < io.M; m0 += a.slots, turn ^= 1) {
    if (R::kAlone && m0 + slot >= io.M) break;
    const bool live = R::kAlone || (used && m0 + slot < io.M);
    const int cols = live ? n : 0;
    float x[E], z[E], r[E], d[E], dr[E], w[E];
    if (!kAhead) ask(m0);
    if (after || gate || scale) rx.get(x);
    if (gate) rz.get(z);
    if (weight) rdy.get(d), rr.get(r);
    if (from_r) rdr.get(dr);
    if (kAhead && m0 + a.slots < io.M) ask(m0 + a.slots);

    float q[K] = {};
    if constexpr (S > 0) if (weight) {
      weights(A, io.weight, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[0] = fmaf(r[e], r[e], q[0]);
        q[1] = fmaf(d[e] * w[e], r[e], q[1]);
      }
    }
    if constexpr (A > 0) if (after) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[K - 1] = fmaf(x[e], x[e], q[K - 1]);
    }
    if (weight || after) row_sums<TPR>(q, part1[turn]);
    if (!weight) {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = dr[e];
    } else if constexpr (S > 0) {
      const float i = live ? rsqrtf(fmaf(q[0], rn, io.eps)) : 0.f, c = i * (q[1] * rn);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[e] *= i;
      }
      sum_weight.add(d, r);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = i * fmaf(d[e], w[e], -(r[e] * c));
      if (from_r) {
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] += dr[e];
      }
    }
    if (a.dres) R::store(dres, t, cols, d), dres += step;
    if (!(after || gate || scale)) {
      if (a.dx) R::store(dx, t, cols, d), dx += step;
      continue;
    }

    float j = 1.f;
    if (after) {
      j = live ? rsqrtf(fmaf(q[K - 1], rn, io.eps)) : 0.f;
      weights(0, io.after, w);
    }
    if (after) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= j;  // the norm before its weight
    }
    float s[E];  // act(gate); z becomes its slope
    if (gate && silu_gate) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float p = sigmoid(z[e]);
        s[e] = z[e] * p;
        z[e] = fmaf(s[e], 1.f - p, p);
      }
    } else if (gate) {
#pragma unroll
      for (int e = 0; e < E; ++e) s[e] = z[e], z[e] = 1.f;
    }
    if (scale) {
      float o[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e] = after ? x[e] * w[e] : x[e];
        if (gate) o[e] *= s[e];
      }
      sum_scale.add(d, o);
      weights(A + S, io.scale, o);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] *= o[e];
    }
    if (gate) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        z[e] *= after ? d[e] * (x[e] * w[e]) : d[e] * x[e];
        d[e] *= s[e];
      }
      if (a.dgate) R::store(dgate, t, cols, z), dgate += step;
    }
    if (after) {
      float g[1] = {0.f};
      sum_after.add(d, x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        d[e] *= w[e];
        g[0] = fmaf(d[e], x[e], g[0]);
      }
      row_sums<TPR>(g, part2[turn]);
      const float c = g[0] * rn;
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = j * fmaf(-c, x[e], d[e]);
    }
    if (a.dx) R::store(dx, t, cols, d), dx += step;
  }
  if (!used) return;
  float* p = a.part + (long long)slot * a.kinds * io.D + off;
  float s[E];
  if (a.dafter) sum_after.get(s), R::store(p, t, n, s), p += io.D;
  if (a.dscale) sum_scale.get(s), R::store(p, t, n, s), p += io.D;
  if (a.dweight) sum_weight.get(s), R::store(p, t, n, s);
}

template <typename TX, typename TR, bool VEC, int KIND>
int launch_rows(const NormBackward& a, cudaStream_t s) {
  return norm_by_width<512, KIND == kStream>(a.io.D / a.io.groups, [&](auto tpr, auto pieces) {
    constexpr int block = norm_block(tpr), RPB = block / int(tpr);
    const long long teams = (long long)a.slots * a.io.groups;
    auto fn = backward_kernel<TX, TR, tpr, pieces, VEC, KIND>;
    constexpr int bytes = shared_sums_bytes(KIND, pieces, block);
    if constexpr (bytes > 0) {
      static PerDevice ready;
      if (ready.get([&] {
            return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? 1 : -1;
          }) < 0)
        return int(SDM_ECUDA);
    }
    fn<<<unsigned((teams + RPB - 1) / RPB), block, bytes, s>>>(a);
    return last_launch_status();
  });
}

}  // namespace

template <typename TX, typename TR>
int launch_norm_backward(const NormBackward& a, int parts, bool vec, cudaStream_t s) {
  return norm_instance(parts, [&](auto kind) {
    return vec ? launch_rows<TX, TR, true, kind>(a, s) : launch_rows<TX, TR, false, kind>(a, s);
  });
}

}  // namespace sdm
