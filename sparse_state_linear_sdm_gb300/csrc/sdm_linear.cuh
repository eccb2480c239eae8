// What the forms of linear attention share (sdm_linear.cu, sdm_linear_tiles.cu).
#pragma once

#include "sdm_layers.cuh"

namespace sdm {

// A sequence in one piece (kWhole); or cut into segments: all but the last reduced to their end states from zero
// (kReduce), then each run from the state in front of it (kJoin).
enum LinearPass { kWhole = 0, kReduce = 1, kJoin = 2 };

// The time limit of the tiles' waits.  Tests only: in this pass and block the copies stop in front of this chunk's load (of the
// slots' order).
struct LinearStall {
  unsigned long long wait_ns = 0;
  int pass = -1, block = 0, chunk = 0, load = 0;
};

struct LinearArgs {
  sdm_linear_args io;
  int vtiles;            // column tiles of v
  int o_dv;              // columns of o as it lies in memory (tiles)
  int segments, segment; // segments of a sequence, tokens of a segment
  float* ws_s;           // [segments][B][H][dk][dv]: each segment's end from zero, then the state in front of it
  float* ws_g;           // [segments][B][H]: sum of g over each segment
  bool vec_qk, vec_v, vec_o; // rows of 16-byte pieces
  bool vec_s;            // rows of the states start on 16 bytes
  int* ws_stop;          // [segments][B][H][vtiles]: whether a wait ran out before the segment's end was known (tiles)
  int* dev_err;
  LinearStall stall;
};

struct Place {
  int vt, h, hk, b, seg, slot;
  int t_lo, t_hi;  // the segment
  int t_end;       // end of its tokens that exist
  bool last;
};

// Block -> column tile, head, sequence, segment.
template <int PASS>
__device__ __forceinline__ Place place_of(const LinearArgs& a) {
  const sdm_linear_args& io = a.io;
  Place p;
  unsigned id = blockIdx.x;
  p.vt = int(id % unsigned(a.vtiles));
  id /= unsigned(a.vtiles);
  p.h = int(id % unsigned(io.H));
  id /= unsigned(io.H);
  p.b = int(id % unsigned(io.B));
  p.seg = int(id / unsigned(io.B));
  p.hk = p.h / (io.H / io.Hk);
  p.slot = row_slot(io.slots, p.b, io.n_slots, a.dev_err);
  const int len = p.slot < 0 ? 0 : row_length(io.lengths, p.b, io.T);
  p.t_lo = PASS == kWhole ? 0 : p.seg * a.segment;
  p.t_hi = PASS == kWhole || io.T - p.t_lo < a.segment ? io.T : p.t_lo + a.segment;  // t_lo + segment may pass 2^31
  p.t_end = min(len, p.t_hi);
  p.last = PASS == kWhole || p.seg == a.segments - 1;
  return p;
}

// The kernel that turns segments' ends into the states in front of them.
int launch_front(const LinearArgs& a, cudaStream_t s);

// The tensor cores' form: bf16, dk up to SDM_LINEAR_TILE_D, and multiples of 8, rows on 16 bytes and positive strides, or
// else a workspace of padded_bytes at `pad` for copies that have them.  Segments of its own.
constexpr int kTileColumns = 128;  // of v a CTA takes
inline int tile_columns(int dv) { return (dv + kTileColumns - 1) / kTileColumns; }
void cut_tiles(int B, int T, int H, int dv, int* segments, int* segment);
size_t padded_bytes(int B, int T, int H, int Hk, int dk, int dv);
int launch_tiles(LinearArgs a, void* pad, cudaStream_t s);

}  // namespace sdm
