// Causal differential attention with fp32 arithmetic (fp32 I/O; bf16 I/O under
// LH_ATTN_SIMT=1, the debugging aid of the attention kernels).
//
//   o = A1 v - lam A2 v,  A_m = softmax(q_m k_m^T / sqrt(D/2) + causal mask)
//   dv = (A1 - lam A2)^T do,  dP = do v^T (one product, both maps read it),
//   dS1 = A1 (dP - d1),  dS2 = -lam A2 (dP - d2),  d_m = <do, A_m v>,
//   dq_m = dS_m k_m / sqrt(D/2),  dk_m = dS_m^T q_m / sqrt(D/2),  dlam = -sum d2.
//
// A query that sees one key has A = 1 and dS = 0 exactly: its differences
// dP - d are set to zero rather than left to the rounding of two sums.
//
// Bound by the fp32 FMA pipe. One block per 64-row tile; 256 threads as 16 x 16,
// each with a 4 x 4 piece of a 64 x 64 product, operands in shared memory with
// rows of D + 4 floats, so that both the 16-byte reads along a row (for A B^T)
// and those across it (for A B) go without bank conflicts: 64 FMAs to 12
// shared-memory wavefronts. The softmax runs online in the exp2 domain; both
// maps share the tile's values. The backward recomputes A from the forward's
// row statistics in two kernels, one per query tile (dq) and one per key tile
// (dk, dv; it walks the query tiles of every head that shares the key/value
// head, so shared heads need no atomics either).
//
// Few tiles leave most of the GPU idle and the longest causal row of tiles sets
// the time. Then a cluster of up to 8 blocks shares one tile (split_of): block r
// takes every r-th tile of the walk, leaves its sums in its shared memory, and
// each block adds up an equal share of the rows from all of them, in rank order
// (forward pass: after scaling to the common maximum).
//
// D = 64 keeps two blocks on an SM (128 registers, a few spilled: dk/dv of 1,021
// tokens x 4 heads 105 -> 69 us), and the next tile is on its way while what
// needs the other operand is computed. Forward and backward, 1,021 tokens x 4 heads
// of 64: 186 us; 2 x 4,096 tokens x 8 heads of 64: 5.26 ms, 46 % of the FMA rate (6.51
// with one block and no copies ahead).
#include <cooperative_groups.h>

#include "k_diff.cuh"

namespace lh {
namespace {

constexpr int TS = kDiffTileFP;
constexpr int NT = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int LP = TS + 4;       // row of a 64 x 64 tile
constexpr int kMaxSplit = 8;

namespace cg = cooperative_groups;

// Blocks per tile: as many as the GPU holds at once (two on an SM with D = 64, one
// with D = 128), no more than the longest walk has tiles. 1,021 tokens x 4 heads of
// 64 (68 tiles): 267, 188, 198 us with 2, 4, 8.
int split_of(int D, long long blocks, long long T) {
  int s = 1;
  while (s < kMaxSplit && 2 * s * blocks <= (D == 64 ? 2 : 1) * 148 && 2 * s * TS <= T + TS) s *= 2;
  return s;
}

// The sum over the cluster's blocks of one float4 at the same place of their
// shared memory.
__device__ __forceinline__ float4 sum_ranks(cg::cluster_group& cl, float* p, int ranks) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int r = 0; r < ranks; ++r) {
    const float4 b = *reinterpret_cast<const float4*>(cl.map_shared_rank(p, r));
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  return a;
}
template <typename T>
__device__ __forceinline__ void put4(T* d, const float4& a) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(d) = a;
  } else {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(d);
    h[0] = __floats2bfloat162_rn(a.x, a.y);
    h[1] = __floats2bfloat162_rn(a.z, a.w);
  }
}

__device__ __forceinline__ float lam_of(const void* lam, int h, const float*) { return static_cast<const float*>(lam)[h]; }
__device__ __forceinline__ float lam_of(const void* lam, int h, const __nv_bfloat16*) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(lam)[h]);
}

// rows [r0, r0 + 64) of a [..][ld] matrix, columns 0 .. D-1, into sm[64][D + 4];
// rows past `end` are zero
template <typename T, int D>
__device__ __forceinline__ void stage(float* sm, const T* src, long long ld, int r0, int end) {
  for (int i = threadIdx.x; i < TS * (D / 8); i += NT) {
    const int r = i / (D / 8), c = (i - r * (D / 8)) * 8;
    float x[8];
    if (r0 + r < end) {
      Vec8<T>::load_f32(src + (long long)(r0 + r) * ld + c, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.f;
    }
    float4* d = reinterpret_cast<float4*>(sm + r * (D + 4) + c);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The same, started for fp32 rows (finished by staged()): the walks ask for a tile
// as soon as its place is free, and do what needs the other operand meanwhile.
template <typename T, int D>
__device__ __forceinline__ void stage_ahead(float* sm, const T* src, long long ld, int r0, int end) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int n = 0; n < TS * (D / 4) / NT; ++n) {
      const int i = threadIdx.x + n * NT, r = i / (D / 4), c = (i - r * (D / 4)) * 4, in = r0 + r < end;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(sm + r * (D + 4) + c)),
                   "l"(src + (in ? (long long)(r0 + r) * ld + c : 0)), "r"(in ? 16 : 0)
                   : "memory");
    }
  } else {
    stage<T, D>(sm, src, ld, r0, end);
  }
}
__device__ __forceinline__ void staged() {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// acc[i][j] += sum over K columns of A[ty*4+i][.] B[tx+16j][.]
template <int K, int LD>
__device__ __forceinline__ void mm_nt(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
#pragma unroll 4
  for (int d = 0; d < K; d += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty * 4 + i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(a[i].x, b[j].x, acc[i][j]);
        acc[i][j] = fmaf(a[i].y, b[j].y, acc[i][j]);
        acc[i][j] = fmaf(a[i].z, b[j].z, acc[i][j]);
        acc[i][j] = fmaf(a[i].w, b[j].w, acc[i][j]);
      }
  }
}

// The columns of a W * 16 wide row that thread tx holds: 2 neighbours (W = 2),
// or runs of 4, 64 apart.
template <int W> __device__ __forceinline__ int ncol(int c, int tx) {
  return W == 2 ? tx * 2 + c : (c / 4) * 64 + tx * 4 + (c & 3);
}

// acc[i][c] += sum over 64 rows of P[ty*4+i][.] V[.][ncol(c)]
template <int W, int LD>
__device__ __forceinline__ void mm_nn(const float* P, const float* V, int ty, int tx, float (&acc)[4][W]) {
#pragma unroll 2
  for (int j = 0; j < TS; j += 4) {
    float p[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(P + (ty * 4 + i) * LP + j);
      p[i][0] = t.x; p[i][1] = t.y; p[i][2] = t.z; p[i][3] = t.w;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      float v[W];
      const float* row = V + (j + jj) * LD;
      if (W == 2) {
        const float2 t = *reinterpret_cast<const float2*>(row + tx * 2);
        v[0] = t.x; v[1] = t.y;
      } else {
#pragma unroll
        for (int c = 0; c + 3 < W; c += 4) {
          const float4 t = *reinterpret_cast<const float4*>(row + c * 16 + tx * 4);
          v[c] = t.x; v[(c + 1) % W] = t.y; v[(c + 2) % W] = t.z; v[(c + 3) % W] = t.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < W; ++c) acc[i][c] = fmaf(p[i][jj], v[c], acc[i][c]);
    }
  }
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int W, typename T>
__device__ __forceinline__ void put(T* row, int tx, const float (&v)[W]) {
#pragma unroll
  for (int c = 0; c < W; ++c) {
    if constexpr (sizeof(T) == 4) row[ncol<W>(c, tx)] = v[c];
    else row[ncol<W>(c, tx)] = __float2bfloat16_rn(v[c]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, D == 64 ? 2 : 1) k_diff_fwd_fp(const DiffGeom g, const T* __restrict__ q, const T* __restrict__ k,
                                                    const T* __restrict__ v, const void* lam, const DiffTile* tiles,
                                                    T* __restrict__ o, float* __restrict__ om, float* __restrict__ lse,
                                                    int split, int* err) {
  constexpr int LD = D + 4, W = D / 16, DM = D / 2;
  extern __shared__ __align__(16) float smf[];
  float *Q = smf, *K = Q + TS * LD, *V = K + TS * LD, *P = V + TS * LD;    // P: two maps
  const int rank = blockIdx.x % split;
  int tile, h;
  diff_place(g.oq, blockIdx.x / split, tile, h);
  if (tile >= diff_used(tiles, g, err)) return;           // the whole cluster
  const DiffTile t = tiles[tile];
  const int hk = h / g.G;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = t.w * TS;                                // first row within the sequence
  const T* kb = k + (long long)t.x * g.ldk + (long long)hk * D;
  const T* vb = v + (long long)t.x * g.ldv + (long long)hk * D;
  const float c2 = kLog2e * rsqrtf((float)DM);
  stage<T, D>(Q, q + (long long)t.x * g.ldq + (long long)h * D, g.ldq, r0, t.y);
  float acc[2][4][W], m[2][4], l[2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[u][i] = -INFINITY;
      l[u][i] = 0.f;
#pragma unroll
      for (int c = 0; c < W; ++c) acc[u][i][c] = 0.f;
    }
  if (rank * TS <= r0) stage_ahead<T, D>(K, kb, g.ldk, rank * TS, t.y);
  for (int n0 = rank * TS; n0 <= r0; n0 += split * TS) {
    staged();                                           // K; nobody reads V any more
    stage_ahead<T, D>(V, vb, g.ldv, n0, t.y);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float s[4][4] = {};
      mm_nt<DM, LD>(Q + u * DM, K + u * DM, ty, tx, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = n0 + tx + 16 * j <= r0 + ty * 4 + i ? s[i][j] * c2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
        // key 0 is in every row's first tile, so the running maximum is finite
        const float mn = fmaxf(m[u][i], row_max(mx)), al = exp2f(m[u][i] - mn);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - mn);
          sum += p;
          P[u * TS * LP + (ty * 4 + i) * LP + tx + 16 * j] = p;
        }
        l[u][i] = l[u][i] * al + row_sum(sum);
        m[u][i] = mn;
#pragma unroll
        for (int c = 0; c < W; ++c) acc[u][i][c] *= al;
      }
    }
    staged();            // V; nobody reads K any more (a warp's 8 rows of P are its own)
    if (n0 + split * TS <= r0) stage_ahead<T, D>(K, kb, g.ldk, n0 + split * TS, t.y);
#pragma unroll
    for (int u = 0; u < 2; ++u) mm_nn<W, LD>(P + u * TS * LP, V, ty, tx, acc[u]);
  }
  const float la = lam_of(lam, h, q);
  if (split > 1) {
    cg::cluster_group cl = cg::this_cluster();
    float *A = smf, *M = smf + 2 * TS * LD;       // [2][64][LD] sums, then [4][64]: maxima and sums of both maps
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = ty * 4 + i;
#pragma unroll
        for (int c = 0; c < W; ++c) A[(u * TS + rr) * LD + ncol<W>(c, tx)] = acc[u][i][c];
        if (tx == 0) {
          M[u * TS + rr] = m[u][i];
          M[(2 + u) * TS + rr] = l[u][i];
        }
      }
    cl.sync();
    const int share = TS / split;
    for (int x = threadIdx.x; x < share * (D / 4); x += NT) {
      const int rr = rank * share + x / (D / 4), c = (x % (D / 4)) * 4, r = r0 + rr;
      if (r >= t.y) continue;
      const long long row = t.x + r;
      float4 both[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float mx = -INFINITY, sum = 0.f;
        for (int k = 0; k < split; ++k) mx = fmaxf(mx, *cl.map_shared_rank(M + u * TS + rr, k));
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < split; ++k) {
          // a block that had no tile has maximum -inf and sums of 0: weight 0
          const float w = exp2f(*cl.map_shared_rank(M + u * TS + rr, k) - mx);
          const float4 b = *reinterpret_cast<const float4*>(cl.map_shared_rank(A + (u * TS + rr) * LD + c, k));
          sum = fmaf(w, *cl.map_shared_rank(M + (2 + u) * TS + rr, k), sum);
          a.x = fmaf(w, b.x, a.x); a.y = fmaf(w, b.y, a.y); a.z = fmaf(w, b.z, a.z); a.w = fmaf(w, b.w, a.w);
        }
        const float inv = 1.f / sum;
        // rounded products, so that o is the same whether they are stored or not
        both[u] = make_float4(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv), __fmul_rn(a.z, inv), __fmul_rn(a.w, inv));
        if (om) put4(om + ((row * g.H + h) * 2 + u) * D + c, both[u]);
        if (lse && c == 0) lse[(2LL * h + u) * g.T + row] = mx + log2f(sum);
      }
      put4(o + row * g.ldo + (long long)h * D + c,
           make_float4(both[0].x - la * both[1].x, both[0].y - la * both[1].y, both[0].z - la * both[1].z, both[0].w - la * both[1].w));
    }
    cl.sync();        // nobody leaves while its sums are still read
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= t.y) continue;
    const long long row = t.x + r;
    float a[W], b[W], both[W];
    const float i0 = 1.f / l[0][i], i1 = 1.f / l[1][i];
#pragma unroll
    for (int c = 0; c < W; ++c) {
      a[c] = __fmul_rn(acc[0][i][c], i0);      // rounded: o is the same whether they are stored or not
      b[c] = __fmul_rn(acc[1][i][c], i1);
      both[c] = a[c] - la * b[c];
    }
    put<W>(o + row * g.ldo + (long long)h * D, tx, both);
    if (om) {
      put<W>(om + (row * g.H + h) * 2 * D, tx, a);
      put<W>(om + ((row * g.H + h) * 2 + 1) * D, tx, b);
    }
    if (lse && tx == 0) {
      lse[(2LL * h) * g.T + row] = m[0][i] + log2f(l[0][i]);       // base 2
      lse[(2LL * h + 1) * g.T + row] = m[1][i] + log2f(l[1][i]);
    }
  }
}

// d1, d2 of every row and head; per block, the sum of d2 (for dlam). One warp
// per row.
template <typename T>
__global__ void __launch_bounds__(256) k_diff_delta_fp(const DiffGeom g, const T* __restrict__ dout,
                                                       const float* __restrict__ om, float* __restrict__ delta,
                                                       float* __restrict__ part) {
  __shared__ float ws[8];
  const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lo = g.cu ? min(max(g.cu[0], 0), g.T) : 0, hi = g.cu ? min(max(g.cu[g.B], 0), g.T) : g.T;
  float tot = 0.f;
  for (int r = warp; r < kDiffDeltaRows; r += 8) {
    const long long row = (long long)blockIdx.x * kDiffDeltaRows + r;
    if (row < lo || row >= hi) continue;
    float a = 0.f, b = 0.f;
    for (int c = lane; c < g.D; c += 32) {
      const T* pd = dout + row * g.ldo + (long long)h * g.D + c;
      float d;
      if constexpr (sizeof(T) == 4) d = *pd;
      else d = __bfloat162float(*pd);
      a = fmaf(d, om[(row * g.H + h) * 2 * g.D + c], a);
      b = fmaf(d, om[((row * g.H + h) * 2 + 1) * g.D + c], b);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, s);
      b += __shfl_xor_sync(0xffffffffu, b, s);
    }
    if (lane == 0) {
      delta[(2LL * h) * g.T + row] = a;
      delta[(2LL * h + 1) * g.T + row] = b;
    }
    tot += b;
  }
  if (lane == 0) ws[warp] = tot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += ws[i];
    part[(size_t)h * gridDim.x + blockIdx.x] = s;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, D == 64 ? 2 : 1) k_diff_dq_fp(const DiffGeom g, const T* __restrict__ dout, const T* __restrict__ q,
                                                   const T* __restrict__ k, const T* __restrict__ v, const void* lam,
                                                   const DiffTile* tiles, const float* __restrict__ lse,
                                                   const float* __restrict__ delta, T* __restrict__ dq, int split, int* err) {
  constexpr int LD = D + 4, DM = D / 2, W = DM / 16;
  extern __shared__ __align__(16) float smf[];
  float *Q = smf, *O = Q + TS * LD, *K = O + TS * LD, *V = K + TS * LD, *S = V + TS * LD;
  const int rank = blockIdx.x % split;
  int tile, h;
  diff_place(g.oq, blockIdx.x / split, tile, h);
  if (tile >= diff_used(tiles, g, err)) return;           // the whole cluster
  const DiffTile t = tiles[tile];
  const int hk = h / g.G;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int r0 = t.w * TS;
  const T* kb = k + (long long)t.x * g.ldk + (long long)hk * D;
  const T* vb = v + (long long)t.x * g.ldv + (long long)hk * D;
  const float sc = rsqrtf((float)DM), c2 = kLog2e * sc, la = lam_of(lam, h, q);
  stage<T, D>(Q, q + (long long)t.x * g.ldq + (long long)h * D, g.ldq, r0, t.y);
  stage<T, D>(O, dout + (long long)t.x * g.ldo + (long long)h * D, g.ldo, r0, t.y);
  float ls[2][4], dl[2][4], acc[2][4][W] = {};
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + ty * 4 + i;
      const long long at = (2LL * h + u) * g.T + t.x + r;
      ls[u][i] = r < t.y ? lse[at] : 0.f;
      dl[u][i] = r < t.y ? delta[at] : 0.f;
    }
  if (rank * TS <= r0) stage_ahead<T, D>(V, vb, g.ldv, rank * TS, t.y);
  for (int n0 = rank * TS; n0 <= r0; n0 += split * TS) {
    staged();                                           // V; nobody reads K any more
    stage_ahead<T, D>(K, kb, g.ldk, n0, t.y);
    float dp[4][4] = {};
    mm_nt<D, LD>(O, V, ty, tx, dp);
    staged();                                           // K; nobody reads V any more
    if (n0 + split * TS <= r0) stage_ahead<T, D>(V, vb, g.ldv, n0 + split * TS, t.y);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float s[4][4] = {};
      mm_nt<DM, LD>(Q + u * DM, K + u * DM, ty, tx, s);
      const float f = u ? -la * sc : sc;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = r0 + ty * 4 + i;
          const bool in = n0 + tx + 16 * j <= r && r > 0;      // row 0 sees one key: dS = 0
          S[u * TS * LP + (ty * 4 + i) * LP + tx + 16 * j] =
              in ? exp2f(fmaf(s[i][j], c2, -ls[u][i])) * (dp[i][j] - dl[u][i]) * f : 0.f;
        }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 2; ++u) mm_nn<W, LD>(S + u * TS * LP, K + u * DM, ty, tx, acc[u]);
  }
  if (split > 1) {
    cg::cluster_group cl = cg::this_cluster();
    float* A = smf;                                 // [64][LD]
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < W; ++c) A[(ty * 4 + i) * LD + u * DM + ncol<W>(c, tx)] = acc[u][i][c];
    cl.sync();
    const int share = TS / split;
    for (int x = threadIdx.x; x < share * (D / 4); x += NT) {
      const int rr = rank * share + x / (D / 4), c = (x % (D / 4)) * 4;
      if (r0 + rr < t.y) put4(dq + (t.x + (long long)(r0 + rr)) * g.ldq + (long long)h * D + c, sum_ranks(cl, A + rr * LD + c, split));
    }
    cl.sync();
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    if (r >= t.y) continue;
    T* dst = dq + (t.x + (long long)r) * g.ldq + (long long)h * D;
    put<W>(dst, tx, acc[0][i]);
    put<W>(dst + DM, tx, acc[1][i]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, D == 64 ? 2 : 1) k_diff_dkdv_fp(const DiffGeom g, const T* __restrict__ dout,
                                                     const T* __restrict__ q, const T* __restrict__ k,
                                                     const T* __restrict__ v, const void* lam, const DiffTile* tiles,
                                                     const float* __restrict__ lse, const float* __restrict__ delta,
                                                     T* __restrict__ dk, T* __restrict__ dv, int split, int* err) {
  constexpr int LD = D + 4, DM = D / 2, W = DM / 16, WV = D / 16;
  extern __shared__ __align__(16) float smf[];
  float *K = smf, *V = K + TS * LD, *Q = V + TS * LD, *O = Q + TS * LD, *S = O + TS * LD, *vec = S + TS * LP;
  const int rank = blockIdx.x % split;
  int tile, hk;
  diff_place(g.ok, blockIdx.x / split, tile, hk);
  if (tile >= diff_used(tiles, g, err)) return;           // the whole cluster
  const DiffTile t = tiles[tile];
  const int ntl = (t.y + TS - 1) / TS, jt = ntl - 1 - t.w;      // early key tiles first: they have the most queries
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int k0 = jt * TS;
  const float sc = rsqrtf((float)DM), c2 = kLog2e * sc;
  stage<T, D>(K, k + (long long)t.x * g.ldk + (long long)hk * D, g.ldk, k0, t.y);
  stage<T, D>(V, v + (long long)t.x * g.ldv + (long long)hk * D, g.ldv, k0, t.y);
  float aV[4][WV] = {}, aK[2][4][W] = {};
  {
    // the query tiles from this one on, of every head that shares the key head
    const int per = ntl - jt;
    auto ahead = [&](int it) {
      const int h = hk * g.G + it / per, i0 = k0 + (it % per) * TS;
      stage_ahead<T, D>(Q, q + (long long)t.x * g.ldq + (long long)h * D, g.ldq, i0, t.y);
      // the queries' statistics: lse of both maps, then d of both
      const int u = threadIdx.x >> 6, c = threadIdx.x & 63, in = i0 + c < t.y;
      const long long at = (2LL * h + (u & 1)) * g.T + t.x + i0 + c;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(vec + threadIdx.x)),
                   "l"((u < 2 ? lse : delta) + (in ? at : 0)), "r"(in ? 4 : 0)
                   : "memory");
    };
    if (rank < per * g.G) ahead(rank);
    for (int it = rank; it < per * g.G; it += split) {
      const int h = hk * g.G + it / per, i0 = k0 + (it % per) * TS;
      const float la = lam_of(lam, h, q);
      staged();                                         // Q; nobody reads O any more
      stage_ahead<T, D>(O, dout + (long long)t.x * g.ldo + (long long)h * D, g.ldo, i0, t.y);
      float dp[4][4] = {}, p[4][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float s[4][4] = {};
        mm_nt<DM, LD>(K + u * DM, Q + u * DM, ty, tx, s);
        if (u == 0) {
          staged();                                     // O
          mm_nt<D, LD>(V, O, ty, tx, dp);
        }
        const float f = u ? -la : 1.f;
        __syncwarp();        // the tile's earlier use of S
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int qq = tx + 16 * j, r = i0 + qq;
            const bool in = k0 + ty * 4 + i <= r && r < t.y;
            const float e = in ? exp2f(fmaf(s[i][j], c2, -vec[u * 64 + qq])) * f : 0.f;
            p[i][j] = u ? p[i][j] + e : e;
            S[(ty * 4 + i) * LP + qq] = r > 0 ? e * (dp[i][j] - vec[128 + u * 64 + qq]) * sc : 0.f;
          }
        __syncwarp();
        mm_nn<W, LD>(S, Q + u * DM, ty, tx, aK[u]);
      }
      __syncthreads();                                  // nobody reads Q any more
      if (it + split < per * g.G) ahead(it + split);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[(ty * 4 + i) * LP + tx + 16 * j] = p[i][j];
      __syncwarp();
      mm_nn<WV, LD>(S, O, ty, tx, aV);
    }
  }
  if (split > 1) {
    cg::cluster_group cl = cg::this_cluster();
    float *A = smf, *B = smf + TS * LD;             // dk, dv: [64][LD] each
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < W; ++c) A[(ty * 4 + i) * LD + u * DM + ncol<W>(c, tx)] = aK[u][i][c];
#pragma unroll
      for (int c = 0; c < WV; ++c) B[(ty * 4 + i) * LD + ncol<WV>(c, tx)] = aV[i][c];
    }
    cl.sync();
    const int share = TS / split;
    for (int x = threadIdx.x; x < share * (D / 4); x += NT) {
      const int rr = rank * share + x / (D / 4), c = (x % (D / 4)) * 4;
      if (k0 + rr >= t.y) continue;
      const long long row = t.x + k0 + rr;
      put4(dk + row * g.ldk + (long long)hk * D + c, sum_ranks(cl, A + rr * LD + c, split));
      put4(dv + row * g.ldv + (long long)hk * D + c, sum_ranks(cl, B + rr * LD + c, split));
    }
    cl.sync();
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = k0 + ty * 4 + i;
    if (r >= t.y) continue;
    const long long row = t.x + r;
    put<W>(dk + row * g.ldk + (long long)hk * D, tx, aK[0][i]);
    put<W>(dk + row * g.ldk + (long long)hk * D + DM, tx, aK[1][i]);
    put<WV>(dv + row * g.ldv + (long long)hk * D, tx, aV[i]);
  }
}

// a cluster of `split` blocks per tile and head
template <typename K, typename... A>
cudaError_t launch_split(K kern, int ntile, int heads, int split, int sm, int* err, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)ntile * heads * split);
  c.blockDim = dim3(NT);
  c.dynamicSmemBytes = sm;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&c, kern, args..., split, err);
}

template <typename T, int D>
cudaError_t fwd_t(const DiffGeom& g, const void* q, const void* k, const void* v, const void* lam, const DiffTile* tiles,
                  void* o, float* om, float* lse, int* err, cudaStream_t s) {
  const int sm = (3 * TS * (D + 4) + 2 * TS * LP) * 4;
  auto kern = k_diff_fwd_fp<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
  if (e != cudaSuccess) return e;
  return launch_split(kern, g.ntile, g.H, split_of(D, (long long)g.ntile * g.H, g.T), sm, err, s, g, (const T*)q, (const T*)k, (const T*)v, lam,
                      tiles, (T*)o, om, lse);
}

template <typename T, int D>
cudaError_t bwd_t(const DiffGeom& g, const void* dout, const void* q, const void* k, const void* v, const void* lam,
                  const DiffTile* tiles, const float* lse, const float* delta, void* dq, void* dk, void* dv, int* err,
                  cudaStream_t s) {
  const int sm1 = (4 * TS * (D + 4) + 2 * TS * LP) * 4, sm2 = (4 * TS * (D + 4) + TS * LP + 256) * 4;
  auto kq = k_diff_dq_fp<T, D>;
  auto kk = k_diff_dkdv_fp<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, sm1);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, sm2);
  if (e != cudaSuccess) return e;
  e = launch_split(kk, g.ntile, g.Hk, split_of(D, (long long)g.ntile * g.Hk, (long long)g.T * g.G), sm2, err, s, g, (const T*)dout, (const T*)q,
                   (const T*)k, (const T*)v, lam, tiles, lse, delta, (T*)dk, (T*)dv);
  if (e != cudaSuccess) return e;
  return launch_split(kq, g.ntile, g.H, split_of(D, (long long)g.ntile * g.H, g.T), sm1, err, s, g, (const T*)dout, (const T*)q, (const T*)k,
                      (const T*)v, lam, tiles, lse, delta, (T*)dq);
}

}  // namespace

cudaError_t launch_diff_fwd_fp(const DiffGeom& g, lh_dtype dt, const void* q, const void* k, const void* v,
                               const void* lam, const DiffTile* tiles, void* o, float* om, float* lse, int* err,
                               cudaStream_t s) {
  if (dt == LH_BF16)
    return g.D == 64 ? fwd_t<__nv_bfloat16, 64>(g, q, k, v, lam, tiles, o, om, lse, err, s)
                     : fwd_t<__nv_bfloat16, 128>(g, q, k, v, lam, tiles, o, om, lse, err, s);
  return g.D == 64 ? fwd_t<float, 64>(g, q, k, v, lam, tiles, o, om, lse, err, s)
                   : fwd_t<float, 128>(g, q, k, v, lam, tiles, o, om, lse, err, s);
}

cudaError_t launch_diff_bwd_fp(const DiffGeom& g, lh_dtype dt, const void* dout, const void* q, const void* k,
                               const void* v, const void* lam, const DiffTile* tiles, const float* om,
                               const float* lse, float* delta, float* part, void* dq, void* dk, void* dv, void* dlam,
                               int* err, cudaStream_t s) {
  const int nb = (g.T + kDiffDeltaRows - 1) / kDiffDeltaRows;
  const dim3 gd(nb, g.H);
  if (dt == LH_BF16)
    k_diff_delta_fp<<<gd, 256, 0, s>>>(g, (const __nv_bfloat16*)dout, om, delta, part);
  else
    k_diff_delta_fp<<<gd, 256, 0, s>>>(g, (const float*)dout, om, delta, part);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if ((e = launch_diff_dlam(g.H, nb, part, dt, dlam, s)) != cudaSuccess) return e;
  if (dt == LH_BF16)
    return g.D == 64 ? bwd_t<__nv_bfloat16, 64>(g, dout, q, k, v, lam, tiles, lse, delta, dq, dk, dv, err, s)
                     : bwd_t<__nv_bfloat16, 128>(g, dout, q, k, v, lam, tiles, lse, delta, dq, dk, dv, err, s);
  return g.D == 64 ? bwd_t<float, 64>(g, dout, q, k, v, lam, tiles, lse, delta, dq, dk, dv, err, s)
                   : bwd_t<float, 128>(g, dout, q, k, v, lam, tiles, lse, delta, dq, dk, dv, err, s);
}

}  // namespace lh
