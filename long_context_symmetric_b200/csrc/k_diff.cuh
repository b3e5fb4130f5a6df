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

struct DiffGeom {
  int B, T, H, Hk, G, D;          // G = H / Hk query heads to a key/value head
  int N;                          // rows per sequence when cu is NULL
  long long ldq, ldk, ldv, ldo;   // elements between token rows
  const int* cu;                  // device offsets [B + 1], or NULL
  int ntile;                      // entries of the tile table
  int tag;                        // of the problem that the tile table belongs to
};

// One entry: first row, rows, padded first row, tile index within the sequence.
// tiles[ntile] holds the number of entries that are in use and the problem's tag.
using DiffTile = int4;

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
