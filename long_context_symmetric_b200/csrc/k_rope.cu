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
// Bound by HBM: q and k are read once and written once. A block takes kTok
// tokens: its threads first issue the loads of the first batch of rows, then
// form the tokens' cosines and sines (one per pair, shared by all heads) in
// shared memory while those are under way, then rotate and store. W elements
// to a load: 16 bytes for bf16 when the rows allow it (W = 8), down to single
// elements for row lengths, strides or rotated widths of odd size.
#include "lh_common.cuh"

namespace lh {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kTok = 4;               // tokens per block
constexpr int kBatch = 4;             // items in flight per thread

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  const void* pos;
  const double* freq;
  const int* axis;
  long long tokens;                   // B * N
  int N, H, Hk, D, R, axes;           // R = rot / 2 pairs
  long long q_ld, q_bs, k_ld, k_bs, qo_ld, qo_bs, ko_ld, ko_bs, pos_as, pos_bs;
  int next, pos64, inverse, tail;     // tail: copy the elements behind the rotated ones
  int* err;
};

template <typename T, int W> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> { using V = uint4; };
template <> struct Pack<__nv_bfloat16, 4> { using V = uint2; };
template <> struct Pack<__nv_bfloat16, 2> { using V = uint32_t; };
template <> struct Pack<__nv_bfloat16, 1> { using V = uint16_t; };
struct alignas(16) F8 { float4 a, b; };
template <> struct Pack<float, 8> { using V = F8; };
template <> struct Pack<float, 4> { using V = float4; };
template <> struct Pack<float, 2> { using V = float2; };
template <> struct Pack<float, 1> { using V = float; };

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float& x) { x = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& x) { x = __float2bfloat16_rn(v); }

template <typename T, int W>
union Chunk {
  typename Pack<T, W>::V v;
  T e[W];
  __device__ Chunk() {}
};

// One item: 2 W elements of one row: W pairs (the two halves' vectors, or two
// neighbouring vectors), or two vectors of the tail.
struct Item {
  const char* src;
  char* dst;
  int o0, o1;        // element offsets of the two vectors (o1 < 0: none)
  int pair;          // first pair, or -1: copied as it is
  int tok;           // token within the block
};

template <typename T, int W>
__device__ __forceinline__ bool make_item(const RopeArgs& a, long long tok0, int n, int per_row, int rot_items, int rows, int x,
                                          Item& it) {
  if (x >= n) return false;
  const int row = x / per_row, c = x - row * per_row;
  it.tok = row / rows;
  const int h = row - it.tok * rows;
  const long long g = tok0 + it.tok, b = g / a.N, t = g - b * a.N;
  const bool isq = h < a.H;
  it.src = static_cast<const char*>(isq ? a.q : a.k) +
           sizeof(T) * (isq ? b * a.q_bs + t * a.q_ld + (long long)h * a.D : b * a.k_bs + t * a.k_ld + (long long)(h - a.H) * a.D);
  it.dst = static_cast<char*>(isq ? a.qo : a.ko) +
           sizeof(T) * (isq ? b * a.qo_bs + t * a.qo_ld + (long long)h * a.D : b * a.ko_bs + t * a.ko_ld + (long long)(h - a.H) * a.D);
  if (c < rot_items) {
    it.pair = c * W;
    it.o0 = a.next ? 2 * it.pair : it.pair;
    it.o1 = a.next ? it.o0 + W : it.pair + a.R;
  } else {
    it.pair = -1;
    it.o0 = 2 * a.R + (c - rot_items) * 2 * W;
    it.o1 = it.o0 + W < a.D ? it.o0 + W : -1;
  }
  return true;
}

template <typename T, int W>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const RopeArgs a) {
  extern __shared__ float2 cs[];                       // [kTok][R]: cosine, sine
  using V = typename Pack<T, W>::V;
  const long long tok0 = (long long)blockIdx.x * kTok;
  const int nt = (int)min((long long)kTok, a.tokens - tok0);
  const int rot_items = a.R / W, tail_items = a.tail ? (a.D - 2 * a.R + 2 * W - 1) / (2 * W) : 0;
  const int per_row = rot_items + tail_items, rows = a.H + a.Hk, n = nt * rows * per_row;
  bool ready = false;
  for (int x0 = threadIdx.x; x0 < n || !ready; x0 += kRopeThreads * kBatch) {
    Chunk<T, W> u[kBatch], w[kBatch];
    Item it[kBatch];
    bool in[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      in[k] = make_item<T, W>(a, tok0, n, per_row, rot_items, rows, x0 + k * kRopeThreads, it[k]);
      if (in[k]) {
        const T* s = reinterpret_cast<const T*>(it[k].src);
        u[k].v = *reinterpret_cast<const V*>(s + it[k].o0);
        if (it[k].o1 >= 0) w[k].v = *reinterpret_cast<const V*>(s + it[k].o1);
      }
    }
    if (!ready) {
      for (int y = threadIdx.x; y < nt * a.R; y += kRopeThreads) {
        const int tk = y / a.R, i = y - tk * a.R;
        const long long g = tok0 + tk, b = g / a.N, t = g - b * a.N;
        int ax = __ldg(a.axis + i);
        if (ax < 0 || ax >= a.axes) {
          report_error(a.err, LH_ERR_DEVICE, 401);
          ax = 0;
        }
        const long long at = b * a.pos_bs + ax * a.pos_as + t;
        const double p = a.pos64 ? (double)static_cast<const long long*>(a.pos)[at] : (double)static_cast<const int*>(a.pos)[at];
        // quarter turns: 4 angle / (2 pi) = q + r, |r| <= 1/2
        const double turns = p * (__ldg(a.freq + i) * 0.63661977236758134308);
        const double qd = rint(turns);
        float s, c;
        sincospif((float)((turns - qd) * 0.5), &s, &c);
        const int q4 = (int)((long long)qd & 3);
        const float cc = (q4 & 1) ? s : c, ss = (q4 & 1) ? c : s;
        const float co = (q4 == 1 || q4 == 2) ? -cc : cc, si = q4 >= 2 ? -ss : ss;
        cs[y] = make_float2(co, a.inverse ? -si : si);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!in[k]) continue;
      T* d = reinterpret_cast<T*>(it[k].dst);
      if (it[k].pair >= 0) {
        const float2* c = cs + it[k].tok * a.R + it[k].pair;
        if (a.next && W > 1) {
          // pairs of neighbours: elements (0, 1), (2, 3) .. of u, then of w
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const float2 c0 = c[e / 2], c1 = c[(W + e) / 2];
            const float x0_ = to_f(u[k].e[e]), y0_ = to_f(u[k].e[e + (W > 1)]);
            const float x1_ = to_f(w[k].e[e]), y1_ = to_f(w[k].e[e + (W > 1)]);
            from_f(x0_ * c0.x - y0_ * c0.y, u[k].e[e]);
            from_f(y0_ * c0.x + x0_ * c0.y, u[k].e[e + (W > 1)]);
            from_f(x1_ * c1.x - y1_ * c1.y, w[k].e[e]);
            from_f(y1_ * c1.x + x1_ * c1.y, w[k].e[e + (W > 1)]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float2 c0 = c[e];
            const float xa = to_f(u[k].e[e]), xb = to_f(w[k].e[e]);
            from_f(xa * c0.x - xb * c0.y, u[k].e[e]);
            from_f(xb * c0.x + xa * c0.y, w[k].e[e]);
          }
        }
      }
      *reinterpret_cast<V*>(d + it[k].o0) = u[k].v;
      if (it[k].o1 >= 0) *reinterpret_cast<V*>(d + it[k].o1) = w[k].v;
    }
  }
}

template <typename T, int W>
cudaError_t rope_t(const RopeArgs& a, cudaStream_t st) {
  const long long blocks = (a.tokens + kTok - 1) / kTok;
  const size_t sm = (size_t)kTok * a.R * sizeof(float2);
  k_rope<T, W><<<(unsigned)blocks, kRopeThreads, sm, st>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t rope_w(const RopeArgs& a, int w, cudaStream_t st) {
  switch (w) {
    case 8: return rope_t<T, 8>(a, st);
    case 4: return rope_t<T, 4>(a, st);
    case 2: return rope_t<T, 2>(a, st);
    default: return rope_t<T, 1>(a, st);
  }
}

}  // namespace

cudaError_t launch_rope(const lh_rope_config& c, const void* q, const void* k, const void* pos, const double* freq,
                        const int32_t* axis, int inverse, void* qo, void* ko, int* err, cudaStream_t st) {
  RopeArgs a{};
  a.q = q; a.k = k; a.qo = qo; a.ko = ko; a.pos = pos; a.freq = freq; a.axis = axis; a.err = err;
  a.tokens = (long long)c.B * c.N;
  if (a.tokens == 0) return cudaSuccess;
  a.N = c.N; a.H = c.H; a.Hk = c.Hk; a.D = c.D; a.R = c.rot / 2; a.axes = c.axes;
  const long long wq = (long long)c.H * c.D, wk = (long long)c.Hk * c.D;
  a.q_ld = c.q_ld ? c.q_ld : wq; a.qo_ld = c.qo_ld ? c.qo_ld : wq;
  a.k_ld = c.k_ld ? c.k_ld : wk; a.ko_ld = c.ko_ld ? c.ko_ld : wk;
  a.q_bs = c.q_bs ? c.q_bs : a.q_ld * c.N; a.qo_bs = c.qo_bs ? c.qo_bs : a.qo_ld * c.N;
  a.k_bs = c.k_bs ? c.k_bs : a.k_ld * c.N; a.ko_bs = c.ko_bs ? c.ko_bs : a.ko_ld * c.N;
  a.pos_as = c.pos_as; a.pos_bs = c.pos_bs;
  a.next = c.pairs == LH_ROPE_NEXT; a.pos64 = c.pos64; a.inverse = inverse;
  const bool inplace = q == qo && k == ko && a.q_ld == a.qo_ld && a.q_bs == a.qo_bs && (!c.Hk || (a.k_ld == a.ko_ld && a.k_bs == a.ko_bs));
  a.tail = !inplace && c.rot < c.D;
  // the widest vector that every row start, both halves' starts and the tail's
  // start are multiples of
  const long long all = (long long)c.D | a.R | a.q_ld | a.q_bs | a.k_ld | a.k_bs | a.qo_ld | a.qo_bs | a.ko_ld | a.ko_bs;
  const int w = all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
  return c.dtype == LH_BF16 ? rope_w<__nv_bfloat16>(a, w, st) : rope_w<float>(a, w, st);
}

}  // namespace lh
