// Layer norm of the rows of a matrix, forward and backward, with the reduction
// of the weight's and the bias's gradient.
//
//   z = (x - mean) rstd,  y = z w + b,        rstd = 1 / sqrt(var + eps)
//   g = dy w,  dx = rstd (g - mean(g) - z mean(g z)),
//   dw = sum over rows of dy z,  db = sum over rows of dy
//
// Everything is summed in fp32 and rounded once on the way out; the variance is
// formed from the centred values (a second pass over the registers, not over
// memory), so a row whose mean is far above its deviation keeps its digits.
//
// Bound by HBM: x is read and y written once; the backward reads x and dy and
// writes dx once. A row is held in registers by a group of threads, 8 values to
// a vector: G = 4 .. 32 lanes of a warp for rows of up to 256 values (several rows
// to a warp, sums by shuffles alone), a block for longer ones (one barrier per
// reduction, the partial sums alternating between two buffers); the forward pass
// of bf16 rows of up to 2,048 values takes a warp per row, with no barrier. The
// blocks, but for those, stay resident and walk the rows with a stride, R rows at
// a time and the next R on their way meanwhile, so that the weights are loaded
// once; the backward keeps its columns' dw and db in registers (in shared memory
// for rows of more than 8,192 values, where 512 threads hold 32 columns each and
// the registers do not suffice) and writes one partial row per block, which a
// second kernel adds in a fixed order: no atomics, the same bits every run. Which
// form a row takes goes by its length, type and alignment, never by the number of
// rows, so a row has the same bits in any batch. Arithmetic goes in packed pairs.
//
// Measured: 98,304 rows of 2,048 bf16 149 us forward (5.4 TB/s), 222 us backward
// (5.4), 4 us the sums, of fp32 296 (5.4) and 367 (6.6); 1,048,576 of 128 bf16 99 us
// (5.4) and 134 us (6.0); 5,003 of 1,537 fp32 19 and 33 us. 8,192 of 16,384 bf16 125 us
// forward (4.3), but 606 backward (1.3): the columns' sums in shared memory.
//
// Rows of odd length, or whose stride is no multiple of 8 elements, are read
// element by element with the columns dealt out to neighbouring lanes (VEC =
// false), which keeps the accesses of a warp contiguous.
#include <atomic>

#include "lh_common.cuh"

namespace lh {
namespace {

constexpr int kNormThreads = 512;      // threads that hold one long row at most
constexpr int kRowThreads = 64, kRowBlocks = 10;   // forward pass of a row per warp

struct NormArgs {
  const void *x, *w, *b, *dy;
  void *y, *dx;
  float *mean, *rstd, *part;
  long long M, ldx, ldy;
  int d, wbf16;
  float eps, inv_d;
};

__device__ __forceinline__ void st_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The 8 columns that thread t of a group of `gs` holds in its vector v:
// neighbours (VEC), or one of every gs. Columns past d read as 0.
template <bool VEC>
__device__ __forceinline__ int col_of(int v, int i, int t, int gs) {
  return VEC ? (v * gs + t) * 8 + i : (v * 8 + i) * gs + t;
}
// As they come from memory (a row that is on its way takes no more registers
// than its bytes), and widened.
template <typename T, bool VEC> struct Cols;
template <> struct Cols<__nv_bfloat16, true> {
  uint4 r;
  __device__ void load(const __nv_bfloat16* row, int v, int t, int gs, int d) {
    const int c = (v * gs + t) * 8;
    r = c < d ? __ldg(reinterpret_cast<const uint4*>(row + c)) : make_uint4(0, 0, 0, 0);
  }
  __device__ float get(int i) const {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
template <> struct Cols<float, true> {
  float4 a, b;
  __device__ void load(const float* row, int v, int t, int gs, int d) {
    const int c = (v * gs + t) * 8;
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < d) {
      a = __ldg(reinterpret_cast<const float4*>(row + c));
      b = __ldg(reinterpret_cast<const float4*>(row + c) + 1);
    }
  }
  __device__ float get(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
};
template <typename T> struct Cols<T, false> {
  T x[8];
  __device__ void load(const T* row, int v, int t, int gs, int d) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(v, i, t, gs);
      if (c < d) x[i] = row[c];
      else st_f32(&x[i], 0.f);
    }
  }
  __device__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return x[i];
    else return __bfloat162float(x[i]);
  }
};
template <typename T, bool VEC>
__device__ __forceinline__ void store_cols(T* row, int v, int t, int gs, int d, const float (&x)[8]) {
  if (VEC) {
    const int c = (v * gs + t) * 8;
    if (c < d) Vec8<T>::store_f32(row + c, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<false>(v, i, t, gs);
      if (c < d) st_f32(row + c, x[i]);
    }
  }
}
// Arithmetic goes in pairs (packed fp32 instructions): columns 2 i and 2 i + 1 of
// a vector.
template <typename C> __device__ __forceinline__ float2 pair_of(const C& c, int i) {
  return make_float2(c.get(2 * i), c.get(2 * i + 1));
}
__device__ __forceinline__ float2 pair_of(const float (&x)[8], int i) { return make_float2(x[2 * i], x[2 * i + 1]); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
// -mean, for columns past d 0 (they were read as 0, so their z is 0): one test
// per vector of neighbours
template <bool VEC>
__device__ __forceinline__ float2 neg_mean(float mu, int v, int i, int t, int gs, int d) {
  if (VEC) return both((v * gs + t) * 8 < d ? -mu : 0.f);
  return make_float2(col_of<false>(v, 2 * i, t, gs) < d ? -mu : 0.f, col_of<false>(v, 2 * i + 1, t, gs) < d ? -mu : 0.f);
}

// weight or bias columns (NULL: the given constant)
template <bool VEC>
__device__ __forceinline__ void load_w(const void* w, int bf16, float none, int v, int t, int gs, int d,
                                       float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = none;
  } else if (bf16) {
    Cols<__nv_bfloat16, VEC> c;
    c.load(static_cast<const __nv_bfloat16*>(w), v, t, gs, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c.get(i);
  } else {
    Cols<float, VEC> c;
    c.load(static_cast<const float*>(w), v, t, gs, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c.get(i);
  }
}

// Sum of each of n values over the threads of a row's group. G > 0: lanes of a
// warp. G = 0: the block, through red (32 * n floats; the caller alternates
// between two of them, so one barrier per reduction suffices: a buffer is
// written again only after the other one's barrier).
template <int G, int n>
__device__ __forceinline__ void group_sum(float (&v)[n], float* red) {
#pragma unroll
  for (int o = (G ? G : 32) / 2; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
  if (G == 0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < n; ++k) red[warp * n + k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = lane < nw ? red[lane * n + k] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
#pragma unroll
      for (int k = 0; k < n; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
  }
}

template <typename T, bool VEC, int G, int NV, int R>
__global__ void __launch_bounds__(G == 0 ? kNormThreads : NV == 1 ? 256 : kRowThreads, G == 0 ? 1 : NV == 1 ? 0 : kRowBlocks)
k_norm_fwd(const NormArgs a) {
  constexpr bool AHEAD = G == 0 || NV == 1;
  __shared__ float red[G ? 1 : 2 * 32 * R];
  const int gs = G ? G : (int)blockDim.x, t = G ? (int)threadIdx.x % G : (int)threadIdx.x;
  const int groups = G ? (int)blockDim.x / G : 1, grp = G ? (int)threadIdx.x / G : 0;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  // w and b in registers for rows of one vector per thread; reloaded from L1 for longer ones
  constexpr bool WREG = NV == 1;
  float w[8], b[8];
  if (WREG) {
    load_w<VEC>(a.w, a.wbf16, 1.f, 0, t, gs, a.d, w);
    load_w<VEC>(a.b, a.wbf16, 0.f, 0, t, gs, a.d, b);
  }
  // the block's rows: `base` is the same for the whole block, so every thread
  // takes part in every reduction. AHEAD: the next R rows are asked for before
  // these are worked on.
  const long long step = (long long)gridDim.x * groups;
  Cols<T, VEC> nx[R][NV];
  auto fetch = [&](long long base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long m = base + r * step + grp;
#pragma unroll
      for (int v = 0; v < NV; ++v) nx[r][v].load(x + (m < a.M ? m : 0) * a.ldx, v, t, gs, m < a.M ? a.d : 0);
    }
  };
  if (AHEAD) fetch((long long)blockIdx.x * groups);
  for (long long base = (long long)blockIdx.x * groups; base < a.M; base += step * R) {
    Cols<T, VEC> xr[R][NV];
    float s[R], mu[R], q[R];
    if (!AHEAD) fetch(base);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int v = 0; v < NV; ++v) xr[r][v] = nx[r][v];
    if (AHEAD && base + step * R < a.M) fetch(base + step * R);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 p = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) p = __fadd2_rn(p, pair_of(xr[r][v], i));
      s[r] = p.x + p.y;
    }
    group_sum<G, R>(s, red);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mu[r] = s[r] * a.inv_d;
      float2 p = both(0.f);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = __fadd2_rn(pair_of(xr[r][v], i), neg_mean<VEC>(mu[r], v, i, t, gs, a.d));
          p = __ffma2_rn(c, c, p);
        }
      q[r] = p.x + p.y;
    }
    group_sum<G, R>(q, red + (G ? 0 : 32 * R));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long m = base + r * step + grp;
      const float rs = 1.f / sqrtf(q[r] * a.inv_d + a.eps);
      if (m < a.M) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float o[8];
          if (!WREG) {
            load_w<VEC>(a.w, a.wbf16, 1.f, v, t, gs, a.d, w);
            load_w<VEC>(a.b, a.wbf16, 0.f, v, t, gs, a.d, b);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 z = __fmul2_rn(__fadd2_rn(pair_of(xr[r][v], i), both(-mu[r])), both(rs));
            const float2 f = __ffma2_rn(z, pair_of(w, i), pair_of(b, i));
            o[2 * i] = f.x;
            o[2 * i + 1] = f.y;
          }
          store_cols<T, VEC>(y + m * a.ldy, v, t, gs, a.d, o);
        }
        if (t == 0) {
          if (a.mean) a.mean[m] = mu[r];
          if (a.rstd) a.rstd[m] = rs;
        }
      }
    }
  }
}

// ACC: dw and db of this thread's columns in registers (false: in shared memory).
template <typename T, bool VEC, int G, int NV, int R, bool ACC>
__global__ void __launch_bounds__(G ? 256 : kNormThreads, G ? 2 : 1) k_norm_bwd(const NormArgs a) {
  extern __shared__ float dyn[];
  __shared__ float red[G ? 1 : 2 * 32 * 2 * R];
  const int gs = G ? G : (int)blockDim.x, t = G ? (int)threadIdx.x % G : (int)threadIdx.x;
  const int groups = G ? (int)blockDim.x / G : 1, grp = G ? (int)threadIdx.x / G : 0;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.dx);
  // w in registers for rows of one vector per thread; reloaded from L1 for longer ones
  constexpr int WREG = NV == 1 ? 1 : 0;
  float w[WREG ? NV : 1][8];
  float2 dw[ACC ? NV : 1][4], db[ACC ? NV : 1][4];
  if (WREG) {
#pragma unroll
    for (int v = 0; v < NV; ++v) load_w<VEC>(a.w, a.wbf16, 1.f, v, t, gs, a.d, w[WREG ? v : 0]);
  }
  if (ACC) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) dw[ACC ? v : 0][i] = db[ACC ? v : 0][i] = both(0.f);
  } else {
    for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) dyn[c] = 0.f;
    __syncthreads();
  }
  const long long step = (long long)gridDim.x * groups;
  Cols<T, VEC> nx[R][NV], ny[R][NV];
  float nmu[R], nrs[R];
  auto fetch = [&](long long base) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long m = base + r * step + grp, mm = m < a.M ? m : 0;
      const int d = m < a.M ? a.d : 0;
      nmu[r] = m < a.M ? __ldg(a.mean + mm) : 0.f;
      nrs[r] = m < a.M ? __ldg(a.rstd + mm) : 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        nx[r][v].load(x + mm * a.ldx, v, t, gs, d);
        ny[r][v].load(dy + mm * a.ldy, v, t, gs, d);
      }
    }
  };
  fetch((long long)blockIdx.x * groups);
  int flip = 0;
  for (long long base = (long long)blockIdx.x * groups; base < a.M; base += step * R, flip ^= 1) {
    float2 zv[R][NV][4], gv[R][NV][4];
    float rs[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rs[r] = nrs[r];
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          zv[r][v][i] = __fmul2_rn(__fadd2_rn(pair_of(nx[r][v], i), neg_mean<VEC>(nmu[r], v, i, t, gs, a.d)), both(nrs[r]));
          gv[r][v][i] = pair_of(ny[r][v], i);
        }
    }
    if (base + step * R < a.M) fetch(base + step * R);
    float2 s1[R], s2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) s1[r] = s2[r] = both(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (WREG == 0) load_w<VEC>(a.w, a.wbf16, 1.f, v, t, gs, a.d, w[0]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 z = zv[r][v][i], g = gv[r][v][i];
          if (ACC) {
            dw[ACC ? v : 0][i] = __ffma2_rn(g, z, dw[ACC ? v : 0][i]);
            db[ACC ? v : 0][i] = __fadd2_rn(db[ACC ? v : 0][i], g);
          } else {
            const int c = col_of<VEC>(v, 2 * i, t, gs), e = col_of<VEC>(v, 2 * i + 1, t, gs);
            if (c < a.d) {
              dyn[c] = fmaf(g.x, z.x, dyn[c]);
              dyn[a.d + c] += g.x;
            }
            if (e < a.d) {
              dyn[e] = fmaf(g.y, z.y, dyn[e]);
              dyn[a.d + e] += g.y;
            }
          }
          const float2 gw = __fmul2_rn(g, pair_of(w[WREG ? v : 0], i));
          gv[r][v][i] = gw;
          s1[r] = __fadd2_rn(s1[r], gw);
          s2[r] = __ffma2_rn(gw, z, s2[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[2 * r] = s1[r].x + s1[r].y;
      s[2 * r + 1] = s2[r].x + s2[r].y;
    }
    group_sum<G, 2 * R>(s, red + (G ? 0 : flip * 64 * R));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long m = base + r * step + grp;
      if (m < a.M) {
        const float c1 = s[2 * r] * a.inv_d, c2 = s[2 * r + 1] * a.inv_d;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __fmul2_rn(both(rs[r]), __ffma2_rn(zv[r][v][i], both(-c2), __fadd2_rn(gv[r][v][i], both(-c1))));
            o[2 * i] = f.x;
            o[2 * i + 1] = f.y;
          }
          store_cols<T, VEC>(dx + m * a.ldx, v, t, gs, a.d, o);
        }
      }
    }
  }
  if (!a.part) return;
  float* out = a.part + (size_t)blockIdx.x * 2 * a.d;
  if (!ACC) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) out[c] = dyn[c];
  } else if (G == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col_of<VEC>(v, i, t, gs);
        if (c < a.d) {
          out[c] = i & 1 ? dw[ACC ? v : 0][i / 2].y : dw[ACC ? v : 0][i / 2].x;
          out[a.d + c] = i & 1 ? db[ACC ? v : 0][i / 2].y : db[ACC ? v : 0][i / 2].x;
        }
      }
  } else {
    // the block's groups hold the same columns: add them in group order
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col_of<VEC>(v, i, t, gs);
        if (c < a.d) {
          dyn[(2 * grp) * a.d + c] = i & 1 ? dw[ACC ? v : 0][i / 2].y : dw[ACC ? v : 0][i / 2].x;
          dyn[(2 * grp + 1) * a.d + c] = i & 1 ? db[ACC ? v : 0][i / 2].y : db[ACC ? v : 0][i / 2].x;
        }
      }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < groups; ++k) s += dyn[2 * k * a.d + c];
      out[c] = s;
    }
  }
}

// dw and db: the blocks' partial rows added in block order, 32 columns to a
// block, 32 strands that a fixed tree joins.
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* __restrict__ part, int nb, int d, void* dw,
                                                      void* db, int wbf16) {
  __shared__ float sm[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < 2 * d) {
    const float* p = part + c;
#pragma unroll 4
    for (int k = threadIdx.y; k < nb; k += 32) s += __ldg(p + (size_t)k * 2 * d);
  }
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  float v = sm[threadIdx.x][threadIdx.y];      // column threadIdx.y, strand threadIdx.x
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < 2 * d) {
    void* dst = cc < d ? dw : db;
    const int k = cc < d ? cc : cc - d;
    if (dst) {
      if (wbf16) static_cast<__nv_bfloat16*>(dst)[k] = __float2bfloat16_rn(v);
      else static_cast<float*>(dst)[k] = v;
    }
  }
}

// How a row of d values is dealt out: lanes of a warp up to 256 values, a block
// beyond; nv vectors of 8 per thread.
struct NormShape {
  int G, threads, nv;
};
NormShape norm_shape(int d, bool warp_rows) {
  const int nvec = (d + 7) / 8;
  if (warp_rows && nvec > 32 && nvec <= 256) return {32, 256, nvec <= 64 ? 2 : nvec <= 128 ? 4 : 8};
  if (nvec <= 32) {
    int G = 4;
    while (G < nvec) G *= 2;
    return {G, 256, 1};
  }
  const int nv = nvec <= kNormThreads ? 1 : nvec <= 2 * kNormThreads ? 2 : 4, th = (nvec + nv - 1) / nv;
  return {0, (th + 31) / 32 * 32, nv};
}
constexpr int kNormSMs = 148;
// Resident blocks: as many as the registers allow, 1,024 threads to an SM for rows
// that lanes of a warp hold, 512 for rows that a block holds.
int norm_blocks(const NormShape& s, long long M, int R) {
  const long long groups = s.G ? s.threads / s.G : 1, need = (M + groups * R - 1) / (groups * R);
  const int per_sm = (s.G ? 1024 : 512) / s.threads;
  const long long most = (long long)kNormSMs * (per_sm < 1 ? 1 : per_sm);
  return (int)(need < most ? need : most);
}
constexpr int kRF = 2;               // rows in flight per group, forward pass (nv = 1)

template <typename T, bool VEC>
cudaError_t fwd_t(const NormShape& s, const NormArgs& a, cudaStream_t st) {
  if (s.G == 32 && s.nv > 1) {
    // a warp per row, every row in flight at once
    if constexpr (VEC && sizeof(T) == 2) {
      const int R = s.nv == 2 ? 2 : 1;
      const long long rows = kRowThreads / 32 * R, need = (a.M + rows - 1) / rows;
      const unsigned nb = (unsigned)(need < 0x7fffffff ? need : 0x7fffffff);
      auto kern = s.nv == 2 ? k_norm_fwd<T, VEC, 32, 2, 2> : s.nv == 4 ? k_norm_fwd<T, VEC, 32, 4, 1> : k_norm_fwd<T, VEC, 32, 8, 1>;
      kern<<<nb, kRowThreads, 0, st>>>(a);
    }
  } else {
    const int nb = norm_blocks(s, a.M, s.nv == 1 ? kRF : 1);
    auto kern = s.G == 4    ? k_norm_fwd<T, VEC, 4, 1, kRF>
                : s.G == 8  ? k_norm_fwd<T, VEC, 8, 1, kRF>
                : s.G == 16 ? k_norm_fwd<T, VEC, 16, 1, kRF>
                : s.G == 32 ? k_norm_fwd<T, VEC, 32, 1, kRF>
                : s.nv == 1 ? k_norm_fwd<T, VEC, 0, 1, kRF>
                : s.nv == 2 ? k_norm_fwd<T, VEC, 0, 2, 1>
                            : k_norm_fwd<T, VEC, 0, 4, 1>;
    kern<<<nb, s.threads, 0, st>>>(a);
  }
  count_launch();
  return cudaGetLastError();
}

// Rows in flight of the backward kernel (one vector per thread): what the
// registers hold without spilling. 1M rows of 128 bf16: 147 us with 2, 130 with 3;
// 98,304 of 2,048: 282, 224, 265 with 1, 2, 3; 5,003 odd fp32 rows of 1,537: 34, 41
// with 1, 2.
template <typename T, bool VEC> constexpr int bwd_rows(int G) {
  return !VEC ? 1 : G > 0 && sizeof(T) == 2 ? 3 : 2;
}
int bwd_blocks(const NormShape& s, long long M, bool vec, bool bf16) {
  const int R = s.nv > 1 ? 1 : !vec ? 1 : s.G > 0 && bf16 ? 3 : 2;
  return norm_blocks(s, M, R);
}

template <typename T, bool VEC>
cudaError_t bwd_t(const NormShape& s, const NormArgs& a, int nb, cudaStream_t st) {
  constexpr int RG = bwd_rows<T, VEC>(32), RB = bwd_rows<T, VEC>(0);
  const size_t sm = s.G ? (size_t)(s.threads / s.G) * 2 * a.d * 4 : s.nv == 4 ? (size_t)2 * a.d * 4 : 0;
  auto kern = s.G == 4    ? k_norm_bwd<T, VEC, 4, 1, RG, true>
              : s.G == 8  ? k_norm_bwd<T, VEC, 8, 1, RG, true>
              : s.G == 16 ? k_norm_bwd<T, VEC, 16, 1, RG, true>
              : s.G == 32 ? k_norm_bwd<T, VEC, 32, 1, RG, true>
              : s.nv == 1 ? k_norm_bwd<T, VEC, 0, 1, RB, true>
              : s.nv == 2 ? k_norm_bwd<T, VEC, 0, 2, 1, true>
                          : k_norm_bwd<T, VEC, 0, 4, 1, false>;
  if (s.nv == 4) {
    // The attribute belongs to the kernel on its device, not to this call: it is set
    // once, to what the longest row needs, so that no call takes back what another
    // host thread's is about to launch with.
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (done.load() >> dev & 1))) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * LH_NORM_MAX_D * 4);
      if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    }
    if (e != cudaSuccess) return e;
  }
  kern<<<nb, s.threads, sm, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

bool norm_vec(const lh_norm_config& c, long long ldx, long long ldy) {
  return c.d % 8 == 0 && ldx % 8 == 0 && ldy % 8 == 0;
}

}  // namespace

// Partial rows of dw and db: one of 2 d floats per block of the backward kernel.
size_t norm_ws_bytes(const lh_norm_config& c) {
  const bool vec = norm_vec(c, c.ldx ? c.ldx : c.d, c.ldy ? c.ldy : c.d);
  return (size_t)bwd_blocks(norm_shape(c.d, false), c.M, vec, c.dtype == LH_BF16) * 2 * c.d * sizeof(float);
}

cudaError_t launch_norm_fwd(const lh_norm_config& c, const void* x, const void* w, const void* b, void* y,
                            float* mean, float* rstd, cudaStream_t st) {
  if (c.M == 0) return cudaSuccess;
  NormArgs a{};
  a.x = x; a.w = w; a.b = b; a.y = y; a.mean = mean; a.rstd = rstd;
  a.M = c.M; a.ldx = c.ldx ? c.ldx : c.d; a.ldy = c.ldy ? c.ldy : c.d; a.d = c.d;
  a.wbf16 = c.wdtype == LH_BF16; a.eps = c.eps; a.inv_d = 1.f / (float)c.d;
  const bool vec = norm_vec(c, a.ldx, a.ldy);
  // a warp per row of up to 2,048 bf16 values: 98,304 rows of 2,048 take 150 us
  // against 171 with a block per row; 64 rows of 1,024 take 7.2 against 4.8 (from
  // cold), but by the row count one row would have other bits in another batch
  const NormShape s = norm_shape(c.d, vec && c.dtype == LH_BF16);
  if (c.dtype == LH_BF16)
    return vec ? fwd_t<__nv_bfloat16, true>(s, a, st) : fwd_t<__nv_bfloat16, false>(s, a, st);
  return vec ? fwd_t<float, true>(s, a, st) : fwd_t<float, false>(s, a, st);
}

cudaError_t launch_norm_bwd(const lh_norm_config& c, const void* dy, const void* x, const void* w, const float* mean,
                            const float* rstd, void* dx, void* dw, void* db, float* part, cudaStream_t st) {
  NormArgs a{};
  a.x = x; a.w = w; a.dy = dy; a.dx = dx; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.part = dw || db ? part : nullptr;
  a.M = c.M; a.ldx = c.ldx ? c.ldx : c.d; a.ldy = c.ldy ? c.ldy : c.d; a.d = c.d;
  a.wbf16 = c.wdtype == LH_BF16; a.eps = c.eps; a.inv_d = 1.f / (float)c.d;
  const NormShape s = norm_shape(c.d, false);
  const bool vec = norm_vec(c, a.ldx, a.ldy);
  const int nb = bwd_blocks(s, c.M, vec, c.dtype == LH_BF16);
  if (c.M > 0) {
    cudaError_t e;
    if (c.dtype == LH_BF16)
      e = vec ? bwd_t<__nv_bfloat16, true>(s, a, nb, st) : bwd_t<__nv_bfloat16, false>(s, a, nb, st);
    else
      e = vec ? bwd_t<float, true>(s, a, nb, st) : bwd_t<float, false>(s, a, nb, st);
    if (e != cudaSuccess) return e;
  }
  if (dw || db) {      // no rows: the sums are zero (nb = 0)
    k_norm_reduce<<<(2 * c.d + 31) / 32, dim3(32, 32), 0, st>>>(part, nb, c.d, dw, db, a.wbf16);
    count_launch();
    return cudaGetLastError();
  }
  return cudaSuccess;
}

}  // namespace lh
