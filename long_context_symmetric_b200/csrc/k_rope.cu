// Rotary positions of queries and keys over one or several axes, and the
// inverse rotation (which is the backward pass: a rotation's transpose).
//
// Pair i of a row, (a, b), turns by the angle pos[axis[i]] * freq[i]:
//   a' = a cos - b sin,  b' = b cos + a sin        (inverse: sin negated)
// with the position of the row's token along the pair's axis. The angle is
// formed in 64 bits and reduced there to a quarter turn, so that a position of
// a million keeps every digit of the angle that its cosine needs; cosine, sine
// and the rotation itself are fp32, rounded once on the way out.
//
// Bound by HBM: q and k are read once and written once. A block takes a few
// tokens (kTok, or more where a token has few rows): its threads first issue the
// loads of their first items, then form the tokens' cosines and sines (one per
// pair, shared by all heads) in shared memory while those are under way, then
// rotate and store. W elements to a load: 16 bytes when the rows allow it, down
// to single elements for row lengths, strides or rotated widths of odd size.
// Measured: 524,288 tokens of 32 heads of 128 bf16 1.34 - 1.48 ms from GPU to GPU, 5.8
// - 6.4 TB/s (a plain copy: 6.5); 256 tokens 4.2 us; 2 x 8,191 tokens of 10 heads of 64,
// 48 rotated, fp32 15 us (1,366 blocks on 444 places: the fourth wave runs nearly empty).
#include "lh_common.cuh"

namespace lh {
namespace {

constexpr int kTok = 4;               // tokens per thread, all in flight at once
constexpr int kRopeSmem = 16384;      // cosines and sines of a block's tokens, at most (or of kTok tokens)

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  const void* pos;
  const double* freq;
  const int* axis;
  int B, N, H, Hk, D, R, axes;        // R = rot / 2 pairs
  int per_row, rot_items, rows;       // items of a row, those of its rotated part, rows of a token
  int lanes;                          // groups of kTok tokens to a block
  unsigned long long m_row, m_tok;    // 2^36 / per_row, 2^36 / (rows per_row), rounded up
  long long q_ld, q_bs, k_ld, k_bs, qo_ld, qo_bs, ko_ld, ko_bs, pos_as, pos_bs;
  int next, pos64, inverse;
  int* err;
};
// x / d by the rounded reciprocal m = ceil(2^36 / d): exact while x d < 2^36
__device__ __forceinline__ int div36(int x, unsigned long long m) { return (int)(((unsigned long long)x * m) >> 36); }

template <typename T, int W> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> { using V = uint4; };
template <> struct Pack<__nv_bfloat16, 4> { using V = uint2; };
template <> struct Pack<__nv_bfloat16, 2> { using V = uint32_t; };
template <> struct Pack<__nv_bfloat16, 1> { using V = uint16_t; };
template <> struct Pack<float, 4> { using V = float4; };
template <> struct Pack<float, 2> { using V = float2; };
template <> struct Pack<float, 1> { using V = float; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float& x) { x = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

template <bool S, typename V> __device__ __forceinline__ V ld_once(const V* p) {
  if constexpr (S) return __ldcs(p);
  else return *p;
}
template <bool S, typename V> __device__ __forceinline__ void st_once(V* p, const V& v) {
  if constexpr (S) __stcs(p, v);
  else *p = v;
}

template <typename T, int W>
union Chunk {
  typename Pack<T, W>::V v;
  T e[W];
  __device__ Chunk() {}
};

// An item is 2 W elements of one row: W pairs (the two halves' vectors, or two
// neighbouring vectors), or two vectors of the tail. A thread takes one item of
// kTok neighbouring tokens: the addresses are formed once for all of them.
// STREAM: data beyond what L2 holds is marked to leave it first.
template <typename T, int W, int TH, bool STREAM>
__global__ void __launch_bounds__(TH, 768 / TH) k_rope(const RopeArgs a) {
  extern __shared__ float2 cs[];                       // [tokens][R]: cosine, sine
  using V = typename Pack<T, W>::V;
  const int b = blockIdx.y + blockIdx.z * 65535;
  if (b >= a.B) return;
  const int t0 = blockIdx.x * a.lanes * kTok, items = a.rows * a.per_row;
  const int nt = min(a.lanes * kTok, a.N - t0);
  bool ready = false;
  for (int x = threadIdx.x; x < items * a.lanes || !ready; x += TH) {
    const int grp = a.lanes > 1 ? div36(x, a.m_tok) : 0,      // more than one only below 256 items
               y = x - grp * items, row = div36(y, a.m_row), c = y - row * a.per_row;
    const int tk = grp * kTok, live = x < items * a.lanes ? min(kTok, nt - tk) : 0;
    const bool isq = row < a.H;
    const int h = isq ? row : row - a.H;
    const long long ld = isq ? a.q_ld : a.k_ld, lo = isq ? a.qo_ld : a.ko_ld;
    const bool turn = c < a.rot_items;
    const int pair = c * W;
    const int o0 = turn ? (a.next ? 2 * pair : pair) : 2 * a.R + (c - a.rot_items) * 2 * W;
    const int o1 = turn && !a.next ? pair + a.R : o0 + W;
    const bool two = o1 < a.D;                          // a tail may end with one vector
    const T* src = static_cast<const T*>(isq ? a.q : a.k) + (isq ? b * a.q_bs : b * a.k_bs) + (t0 + tk) * ld + h * a.D;
    T* dst = static_cast<T*>(isq ? a.qo : a.ko) + (isq ? b * a.qo_bs : b * a.ko_bs) + (t0 + tk) * lo + h * a.D;
    Chunk<T, W> u[kTok], w[kTok];
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      if (k < live) {
        u[k].v = ld_once<STREAM>(reinterpret_cast<const V*>(src + k * ld + o0));
        if (two) w[k].v = ld_once<STREAM>(reinterpret_cast<const V*>(src + k * ld + o1));
      }
    }
    if (!ready) {
      for (int z = threadIdx.x; z < nt * a.R; z += TH) {
        const int tok = z / a.R, i = z - tok * a.R;
        int ax = __ldg(a.axis + i);
        if (ax < 0 || ax >= a.axes) {
          report_error(a.err, LH_ERR_DEVICE, 401);
          ax = 0;
        }
        const long long at = b * a.pos_bs + ax * a.pos_as + t0 + tok;
        const double p = a.pos64 ? (double)static_cast<const long long*>(a.pos)[at] : (double)static_cast<const int*>(a.pos)[at];
        // quarter turns: 4 angle / (2 pi) = q + r, |r| <= 1/2
        const double turns = p * (__ldg(a.freq + i) * 0.63661977236758134308);
        const double qd = rint(turns);
        float s, co;
        sincospif((float)((turns - qd) * 0.5), &s, &co);
        const int q4 = (int)((long long)qd & 3);
        const float cc = (q4 & 1) ? s : co, ss = (q4 & 1) ? co : s;
        const float rc = (q4 == 1 || q4 == 2) ? -cc : cc, rs = q4 >= 2 ? -ss : ss;
        cs[z] = make_float2(rc, a.inverse ? -rs : rs);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kTok; ++k) {
      if (k >= live) break;
      if (turn) {
        const float2* p = cs + (tk + k) * a.R + pair;
        if (a.next && W > 1) {
          // pairs of neighbours: elements (0, 1), (2, 3) .. of u, then of w
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const float2 c0 = p[e / 2], c1 = p[(W + e) / 2];
            const float x0 = to_f(u[k].e[e]), y0 = to_f(u[k].e[e + (W > 1)]);
            const float x1 = to_f(w[k].e[e]), y1 = to_f(w[k].e[e + (W > 1)]);
            from_f(x0 * c0.x - y0 * c0.y, u[k].e[e]);
            from_f(y0 * c0.x + x0 * c0.y, u[k].e[e + (W > 1)]);
            from_f(x1 * c1.x - y1 * c1.y, w[k].e[e]);
            from_f(y1 * c1.x + x1 * c1.y, w[k].e[e + (W > 1)]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float xa = to_f(u[k].e[e]), xb = to_f(w[k].e[e]);
            from_f(xa * p[e].x - xb * p[e].y, u[k].e[e]);
            from_f(xb * p[e].x + xa * p[e].y, w[k].e[e]);
          }
        }
      }
      st_once<STREAM>(reinterpret_cast<V*>(dst + k * lo + o0), u[k].v);
      if (two) st_once<STREAM>(reinterpret_cast<V*>(dst + k * lo + o1), w[k].v);
    }
  }
}

template <typename T, int W>
cudaError_t rope_t(RopeArgs a, int tail, cudaStream_t st) {
  a.rot_items = a.R / W;
  a.per_row = a.rot_items + (tail + 2 * W - 1) / (2 * W);
  a.rows = a.H + a.Hk;
  const int items = a.rows * a.per_row;
  // groups of tokens that a block of th threads takes
  auto lanes_of = [&](int th) {
    const int fit = kRopeSmem / (kTok * a.R * (int)sizeof(float2)), groups = (int)((a.N + kTok - 1LL) / kTok);
    int l = th / items;
    l = l < fit ? l : fit;
    l = l < groups ? l : groups;
    return l < 1 ? 1 : l;
  };
  // Small blocks overlap each other's phases best: 512K tokens of 256 items, 64
  // threads 1.34 ms, 256 threads 1.64. The larger ones where 64 threads would have
  // too little to do in their last round (16K tokens of 80 items: 62 % of the lanes
  // busy against 94 %), or where there are too few blocks to fill the GPU (256
  // tokens of 256 items: 8.0 us with 64 threads, 4.2 with 256).
  auto busy = [&](int th) {
    const int n = items * lanes_of(th);
    return (double)n / ((double)((n + th - 1) / th) * th);
  };
  const bool few = a.B * ((a.N + kTok - 1LL) / kTok) < 148 * 4;
  const int th = few || busy(256) > 1.1 * busy(64) ? 256 : 64;
  a.lanes = lanes_of(th);
  a.m_row = ((1ull << 36) + a.per_row - 1) / a.per_row;
  a.m_tok = ((1ull << 36) + items - 1) / items;
  const int toks = a.lanes * kTok;
  const dim3 grid((unsigned)((a.N + toks - 1LL) / toks), a.B < 65535 ? a.B : 65535, (a.B + 65534) / 65535);
  // moved bytes beyond twice L2 (126 MB): 1.41 -> 1.34 ms at 512K tokens of 32
  // heads of 128; below that what was rotated may still be read from L2
  const bool stream = 2.0 * a.B * a.N * a.rows * a.D * sizeof(T) > 2.5e8;
  auto kern = th == 64 ? (stream ? k_rope<T, W, 64, true> : k_rope<T, W, 64, false>)
                       : (stream ? k_rope<T, W, 256, true> : k_rope<T, W, 256, false>);
  kern<<<grid, th, (size_t)toks * a.R * sizeof(float2), st>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const lh_rope_config& c, const void* q, const void* k, const void* pos, const double* freq,
                        const int32_t* axis, int inverse, void* qo, void* ko, int* err, cudaStream_t st) {
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = qo; a.ko = ko; a.pos = pos; a.freq = freq; a.axis = axis; a.err = err;
  if (c.B == 0 || c.N == 0) return cudaSuccess;
  a.B = c.B; a.N = c.N; a.H = c.H; a.Hk = c.Hk; a.D = c.D; a.R = c.rot / 2; a.axes = c.axes;
  const long long wq = (long long)c.H * c.D, wk = (long long)c.Hk * c.D;
  a.q_ld = c.q_ld ? c.q_ld : wq; a.qo_ld = c.qo_ld ? c.qo_ld : wq;
  a.k_ld = c.k_ld ? c.k_ld : wk; a.ko_ld = c.ko_ld ? c.ko_ld : wk;
  a.q_bs = c.q_bs ? c.q_bs : a.q_ld * c.N; a.qo_bs = c.qo_bs ? c.qo_bs : a.qo_ld * c.N;
  a.k_bs = c.k_bs ? c.k_bs : a.k_ld * c.N; a.ko_bs = c.ko_bs ? c.ko_bs : a.ko_ld * c.N;
  a.pos_as = c.pos_as; a.pos_bs = c.pos_bs;
  a.next = c.pairs == LH_ROPE_NEXT; a.pos64 = c.pos64; a.inverse = inverse;
  const bool inplace = q == qo && k == ko && a.q_ld == a.qo_ld && a.q_bs == a.qo_bs && (!c.Hk || (a.k_ld == a.ko_ld && a.k_bs == a.ko_bs));
  const int tail = inplace ? 0 : c.D - c.rot;      // elements that are copied
  // the widest vector, up to 16 bytes, that every row start, both halves' starts
  // and the tail's start are multiples of
  const long long all = (long long)c.D | a.R | a.q_ld | a.q_bs | a.k_ld | a.k_bs | a.qo_ld | a.qo_bs | a.ko_ld | a.ko_bs;
  const int w = all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
  if (c.dtype == LH_BF16) {
    switch (w) {
      case 8: return rope_t<__nv_bfloat16, 8>(a, tail, st);
      case 4: return rope_t<__nv_bfloat16, 4>(a, tail, st);
      case 2: return rope_t<__nv_bfloat16, 2>(a, tail, st);
      default: return rope_t<__nv_bfloat16, 1>(a, tail, st);
    }
  }
  switch (w) {
    case 8:
    case 4: return rope_t<float, 4>(a, tail, st);
    case 2: return rope_t<float, 2>(a, tail, st);
    default: return rope_t<float, 1>(a, tail, st);
  }
}

}  // namespace lh
