// Differential attention: what its kernels share.
//
// Token rows. q, o and their gradients are [T][H][D], k and v [T][Hk][D], T
// rows in all: B sequences of T / B rows, or (cu) sequence b in rows
// cu[b] .. cu[b+1]-1. A head's q and k row holds two maps of D/2 elements.
//
// Tiles. Sequence b's rows are cut into tiles of TS rows from its own first row.
// The tile table lists every tile, late tiles (whose queries see the most keys)
// first, so that the long blocks of a launch start first. Kernels that walk
// from a key tile to the sequence's end mirror the index: tile n - 1 - i.
// Working copies of the rows keep a padded order in which every tile starts at
// a multiple of TS: sequence b at pad(b) = ceil(cu[b] / TS) TS + b TS, which
// leaves room for each sequence's last part-filled tile without a prefix sum
// (ceil(x) + ceil(y) <= ceil(x + y) + 1).
#pragma once

#include "lh_common.cuh"

namespace lh {

// Division by a number that the host knows: floor(x 2^64-th of m), exact for 32-bit x
// and d (m exceeds 2^64 / d by less than 1, so the quotient by less than x / 2^64).
struct DiffDivisor {
  unsigned long long m;           // ceil(2^64 / d); 0 for d = 1
  int d;
  __device__ __forceinline__ int div(int x) const { return m ? (int)__umul64hi((unsigned long long)(unsigned)x, m) : x; }
  static DiffDivisor by(int d) { return {d == 1 ? 0ull : ~0ull / (unsigned)d + 1, d}; }
};
// Groups of `per` heads (of = per * ntile blocks each), `full` of them and a last one
// of `tail` heads.
struct DiffOrder {
  DiffDivisor of, per, tail;
  int full;
};

struct DiffGeom {
  int B, T, H, Hk, G, D;          // G = H / Hk query heads to a key/value head
  int N;                          // rows per sequence when cu is NULL
  long long ldq, ldk, ldv, ldo;   // elements between token rows
  const int* cu;                  // device offsets [B + 1], or NULL
  int ntile;                      // entries of the tile table
  int tag;                        // of the problem that the tile table belongs to
  DiffOrder oq, ok;               // in which order blocks take the tiles of the H and of the Hk heads
};

// One entry: first row, rows, padded first row, tile index within the sequence.
// tiles[ntile] holds the number of entries that are in use and the problem's tag.
using DiffTile = int4;

// The block's place: tile and head. The tiles of `per` heads go together, the long
// ones of all of them first, so that no long walk starts late (head by head, 16
// heads of 8,192 tokens took 1,587 us forward and backward against 1,550, in loops
// too short for the power cap, nine documents of 7,001 tokens 421 against 372). As many heads as their streamed rows
// fit L2 together: beyond it they are read from HBM again and again (8 heads of
// 65,536 tokens, all together: 2 % slower than one by one).
__device__ __forceinline__ void diff_place(const DiffOrder& r, int block, int& rank, int& head) {
  const int group = r.of.div(block), in = block - group * r.of.d;
  const DiffDivisor& w = group == r.full ? r.tail : r.per;
  rank = w.div(in);
  head = group * r.per.d + in - rank * w.d;
}
inline DiffOrder diff_order(int ntile, int heads, int per) {
  return {DiffDivisor::by(ntile * per), DiffDivisor::by(per), DiffDivisor::by(heads % per ? heads % per : 1), heads / per};
}
constexpr double kDiffGroupBytes = 8e7;

// Entries in use; none (and a report) where the buffer was not written for this
// problem, so that no kernel follows a table of something else.
__device__ __forceinline__ int diff_used(const DiffTile* tiles, const DiffGeom& g, int* err) {
  const int4 t = tiles[g.ntile];
  if (t.y == g.tag) return t.x;
  if (threadIdx.x == 0) report_error(err, LH_ERR_DEVICE, 404);
  return 0;
}

constexpr int kDiffTileTC = 128;  // rows per tile of the tensor-core kernels
constexpr int kDiffTileFP = 64;   // of the fp32 kernels

__host__ __device__ __forceinline__ int diff_ntile(int T, int B, int ts) { return (T + ts - 1) / ts + B; }
// Sequences of a call at most: placing a tile takes one look at each.
constexpr int kDiffMaxSeqs = 65536;

// rows [lo, hi) of sequence b, inside [0, T) whatever cu holds
__device__ __forceinline__ void diff_seq(const DiffGeom& g, int b, int& lo, int& hi) {
  if (g.cu) {
    const int c0 = __ldg(g.cu + b), c1 = __ldg(g.cu + b + 1);
    lo = min(max(c0, 0), g.T);
    hi = min(max(c1, lo), g.T);
  } else {
    lo = b * g.N;
    hi = lo + g.N;
  }
}

// seq (NULL: not wanted): the sequence of each entry; amax: [3][B][Hk], set to zero
cudaError_t launch_diff_tiles(const DiffGeom& g, int ts, DiffTile* tiles, int* seq, uint32_t* amax, int* err,
                              cudaStream_t s);
// dlam[h] = -(sum of the n partial sums part[h][..]), rounded to dtype
cudaError_t launch_diff_dlam(int H, int n, const float* part, lh_dtype dt, void* dlam, cudaStream_t s);

// om: both maps' outputs [T][H][2][D], lse (base 2) [H][2][T]; NULL where no backward follows
cudaError_t launch_diff_fwd_fp(const DiffGeom& g, lh_dtype dt, const void* q, const void* k, const void* v,
                               const void* lam, const DiffTile* tiles, void* o, float* om, float* lse, int* err,
                               cudaStream_t s);
cudaError_t launch_diff_bwd_fp(const DiffGeom& g, lh_dtype dt, const void* dout, const void* q, const void* k,
                               const void* v, const void* lam, const DiffTile* tiles, const float* om,
                               const float* lse, float* delta, float* part, void* dq, void* dk, void* dv, void* dlam,
                               int* err, cudaStream_t s);

constexpr int kDiffDeltaRows = 64;   // rows per block of the delta kernel (one partial sum of dlam each)

}  // namespace lh
