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
// 16,384 x 16 groups of 128 with a gate: 80 us, 0.61 of the HBM floor, at 53 % of the issue slots and 24 warps an SM;
// the stream alone, 16,384 x 2048, 68 (0.58).  Rows off 16 bytes are read element by element: everything of 4099 x 1537,
// bf16 with an fp32 stream, takes 55 (0.37).  Beyond 4096 channels the sums live in shared memory (4096 x 8192
// with everything 207 us, 282 in registers that spilled).
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

// What of the gradient an instance knows how to do: all of it, or only the norm of the stream (dy, r, dr to
// dresidual or dx), or only the norm of x and the gate.  The smaller ones need fewer registers.
enum NormKind { kAll = 0, kStream = 1, kInner = 2 };
constexpr int sm_threads(int kind, int pieces) { return pieces > 1 || kind == kAll ? 512 : 768; }  // of an SM, by registers

template <typename TX, typename TR>
int launch_norm_backward(const NormBackward& a, int kind, bool vec, cudaStream_t s);

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
constexpr bool shared_sums(int kind, int pieces) { return kind == kAll && pieces > 1; }
constexpr int shared_sums_bytes(int kind, int pieces, int block) {
  return shared_sums(kind, pieces) ? 3 * 8 * pieces * 4 * block : 0;
}

template <typename TX, typename TR, int TPR, int P, bool VEC, int KIND>
__global__ void __launch_bounds__(norm_block(TPR), sm_threads(KIND, P) / norm_block(TPR))
    backward_kernel(const __grid_constant__ NormBackward a) {
  // Everything of long rows off 16 bytes has no registers left to ask for more at a time (4099 x 1537: 55 us, 64 if it
  // does), short ones have (32768 x 100: 41 and 35).
  typedef Row<TPR, P, VEC, KIND != kAll || TPR <= 32> R;
  constexpr int E = R::E, RPB = norm_block(TPR) / TPR, W = norm_block(TPR) / 32;
  constexpr int K = KIND == kAll ? 3 : KIND == kStream ? 2 : 1;  // sums of the first round; the last one is of x
  constexpr int kWeights = KIND == kAll ? 3 : 1;
  __shared__ float part1[2][W][K], part2[2][W][1];
  __shared__ Kept<R, norm_block(TPR), kWeights> kept;
  const sdm_norm_args& io = a.io;
  const int t = threadIdx.x % TPR, n = io.D / io.groups;
  const unsigned team = blockIdx.x * RPB + threadIdx.x / TPR;
  const unsigned slot = team / unsigned(io.groups), group = team % unsigned(io.groups);
  const bool used = slot < unsigned(a.slots);
  const long long off = (long long)group * n;
  const float rn = 1.0f / float(n);
  const bool weight = KIND != kInner && a.dy, after = KIND != kStream && io.after, gate = KIND != kStream && io.gate,
             scale = KIND == kAll && io.scale;
  allow_next();

  extern __shared__ float4 sums_at[];
  typedef Sum<E, norm_block(TPR), shared_sums(KIND, P)> S;
  S sum_after(sums_at), sum_scale(sums_at + E / 4 * norm_block(TPR)), sum_weight(sums_at + E / 2 * norm_block(TPR));

  // A row as it lies in memory; the next one is asked for while this one is worked on.
  typename R::template Raw<TX> rx, rz, rdy;
  typename R::template Raw<TR> rr, rdr;
  const TX* px = static_cast<const TX*>(io.x) + (after || gate || scale ? slot * io.x_rs + off : 0);
  const TX* pz = static_cast<const TX*>(io.gate) + (gate ? slot * io.gate_rs + off : 0);
  const TX* pdy = static_cast<const TX*>(a.dy) + (weight ? slot * a.dy_rs + off : 0);
  const TR* pr = static_cast<const TR*>(a.r) + (weight ? slot * a.r_rs + off : 0);
  const TR* pdr = static_cast<const TR*>(a.dr) + (a.dr ? slot * a.dr_rs + off : 0);
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
    if (a.dr) rdr.ask(pdr, t, cols), pdr += a.slots * a.dr_rs;
  };
  constexpr bool kAhead = P == 1 || (P == 2 && KIND != kAll);  // otherwise it takes more registers than it gains
  if (kAhead) ask(0);
  const long long at = used ? off : 0;
  const int mine = used ? n : 0;
  auto keep = [&](int which, const void* p) { kept.put(which, p, io.w_dtype, at, t, mine); };
  auto weights = [&](int which, const void* p, float (&w)[E]) { kept.get(which, p, io.w_dtype, at, t, mine, w); };
  constexpr int kAfter = 0, kWeight = KIND == kAll ? 1 : 0, kScale = 2;
  if (after) keep(kAfter, io.after);
  if (weight) keep(kWeight, io.weight);
  if (KIND == kAll && scale) keep(kScale, io.scale);

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
    if (a.dr) rdr.get(dr);
    if (kAhead && m0 + a.slots < io.M) ask(m0 + a.slots);

    float q[K] = {};
    if constexpr (KIND != kInner) if (weight) {
      weights(kWeight, io.weight, w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        q[0] = fmaf(r[e], r[e], q[0]);
        q[1] = fmaf(d[e] * w[e], r[e], q[1]);
      }
    }
    if (after) {
#pragma unroll
      for (int e = 0; e < E; ++e) q[K - 1] = fmaf(x[e], x[e], q[K - 1]);
    }
    if (weight || after) row_sums<TPR>(q, part1[turn]);
    if (KIND == kInner || !weight) {
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = dr[e];
    } else if constexpr (KIND != kInner) {
      const float i = live ? rsqrtf(fmaf(q[0], rn, io.eps)) : 0.f, c = i * (q[1] * rn);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        r[e] *= i;
      }
      sum_weight.add(d, r);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = i * fmaf(d[e], w[e], -(r[e] * c));
      if (a.dr) {
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
      weights(kAfter, io.after, w);
    }
    if (after) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] *= j;  // the norm before its weight
    }
    float s[E];  // act(gate); z becomes its slope
    if (gate && io.act == SDM_ACT_SILU) {
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
      weights(kScale, io.scale, o);
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
int launch_norm_backward(const NormBackward& a, int kind, bool vec, cudaStream_t s) {
  if (kind == kStream) return vec ? launch_rows<TX, TR, true, kStream>(a, s) : launch_rows<TX, TR, false, kStream>(a, s);
  if (kind == kInner) return vec ? launch_rows<TX, TR, true, kInner>(a, s) : launch_rows<TX, TR, false, kInner>(a, s);
  return vec ? launch_rows<TX, TR, true, kAll>(a, s) : launch_rows<TX, TR, false, kAll>(a, s);
}

}  // namespace sdm
