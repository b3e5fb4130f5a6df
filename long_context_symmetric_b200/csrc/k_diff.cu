// Differential attention: the tile table and the gradient of lambda.
#include "k_diff.cuh"

namespace lh {
namespace {

__device__ __forceinline__ int seq_tiles(const DiffGeom& g, int b, int ts) {
  int lo, hi;
  diff_seq(g, b, lo, hi);
  return (hi - lo + ts - 1) / ts;
}

// One block per sequence. The tile with index i of sequence b comes behind all
// tiles with a larger index and behind the tiles with index i of the sequences
// before b: rank = sum over b' of max(0, n_b' - 1 - i) + #{b' < b: n_b' > i}.
__global__ void k_diff_tiles(const DiffGeom g, int ts, DiffTile* tiles, int* seq, uint32_t* amax, int* err) {
  const int b = blockIdx.x;
  int lo, hi;
  diff_seq(g, b, lo, hi);
  if (g.cu && threadIdx.x == 0) {
    const int c0 = g.cu[b], c1 = g.cu[b + 1];
    if (c0 < 0 || c1 < c0 || c1 > g.T) report_error(err, LH_ERR_DEVICE, 402);
  }
  if (amax)
    for (int i = threadIdx.x; i < 3 * g.Hk; i += blockDim.x) amax[((size_t)(i / g.Hk) * g.B + b) * g.Hk + i % g.Hk] = 0;
  const int n = (hi - lo + ts - 1) / ts;
  const int pad = (lo + ts - 1) / ts * ts + b * ts;
  // a warp per tile, its lanes over the sequences
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += blockDim.x >> 5) {
    long long rank = 0;
    if (g.cu) {
      for (int c = lane; c < g.B; c += 32) {
        const int m = seq_tiles(g, c, ts);
        rank += max(0, m - 1 - i) + (c < b && m > i ? 1 : 0);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    } else {
      rank = (long long)g.B * (n - 1 - i) + b;
    }
    if (lane == 0 && rank < g.ntile) {
      tiles[rank] = make_int4(lo, hi - lo, pad, i);
      if (seq) seq[rank] = b;
    }
  }
  if (b == 0) {
    __shared__ int total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    int s = 0;
    for (int c = threadIdx.x; c < g.B; c += blockDim.x) s += seq_tiles(g, c, ts);
    atomicAdd(&total, s);
    __syncthreads();
    if (threadIdx.x == 0) tiles[g.ntile] = make_int4(min(total, g.ntile), g.tag, 0, 0);
  }
}

__global__ void __launch_bounds__(256) k_diff_dlam(int n, const float* __restrict__ part, int bf16, void* dlam) {
  __shared__ double sm[256];
  const int h = blockIdx.x;
  double s = 0;
  for (int i = threadIdx.x; i < n; i += 256) s += (double)part[(size_t)h * n + i];
  sm[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o; o >>= 1) {
    if (threadIdx.x < o) sm[threadIdx.x] += sm[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const double v = n ? -sm[0] : 0.0;
    if (bf16) static_cast<__nv_bfloat16*>(dlam)[h] = __double2bfloat16(v);
    else static_cast<float*>(dlam)[h] = (float)v;
  }
}

}  // namespace

cudaError_t launch_diff_tiles(const DiffGeom& g, int ts, DiffTile* tiles, int* seq, uint32_t* amax, int* err,
                              cudaStream_t s) {
  k_diff_tiles<<<g.B, 256, 0, s>>>(g, ts, tiles, seq, amax, err);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_diff_dlam(int H, int n, const float* part, lh_dtype dt, void* dlam, cudaStream_t s) {
  k_diff_dlam<<<H, 256, 0, s>>>(n, part, dt == LH_BF16, dlam);
  count_launch();
  return cudaGetLastError();
}

}  // namespace lh
