// Differential attention on the tensor cores: buffers and constants that the
// forward and backward kernels share.
#pragma once

#include <atomic>

#include "k_diff.cuh"
#include "tc_ptx.cuh"

namespace lh {

constexpr int kDSub = 128 * 64 * 2;   // one 128-row x 64-column 16-bit swizzle tile

// Parts of the caller's buffers. Padded rows: g.ntile * 128 per head.
struct DiffTC {
  DiffTile* tiles;            // [ntile + 1]
  int* seq;                   // [ntile]: the tile's sequence
  uint32_t* amax;             // [3][B][Hk] largest magnitudes of q (over the query heads that share the
                              // key/value head), k, v
  __half *qs, *ks, *vs;       // [H | Hk][padded rows][D]
  __half* om;                 // [H][2][padded rows][D]: A_m v 2^-ev
  float* lse;                 // [H][2][padded rows], base 2
  int* rowx;                  // [H][padded rows]: row_word of each row of do
  int* tmax;                  // [H][padded tiles]: the largest of both parts in the tile
  __half* dos;                // [H][padded rows][D]: do 2^-e, e of the row
  float* delta;               // [H][2][padded rows]: d_m 2^-(e + ev)
  float* part;                // [H][ntile] sums of A2 dP
};

// The power of two of a working copy: x 2^-e, e = 0 while the head's largest
// magnitude is in [1/8, 256), else what brings it into [4, 8). Wider downwards
// than scale_exp's window, so that values of ordinary size need one pass: with a
// largest value of 1/8, bf16 values down to 2^-14 of it still enter unchanged and
// smaller ones are off by at most 2^-22 of it.
__host__ __device__ __forceinline__ int diff_exp(uint32_t amax_bits) {
  const int ex = (int)((amax_bits >> 23) & 0xFFu) - 127;
  return ex >= -3 && ex < 2 ? 0 : scale_exp(amax_bits);
}

// A row of do: the exponent e of its copy, and x with |row|_1 < 2^x; kRowNone
// where it has nothing to say.
constexpr int kRowNone = -1000;
__device__ __forceinline__ int row_word(int e, int x) { return (int)((unsigned)x << 16 | ((unsigned)e & 0xFFFFu)); }
__device__ __forceinline__ int row_e(int w) { return (short)(w & 0xFFFF); }
__device__ __forceinline__ int row_x(int w) { return w >> 16; }

// Registers. A CTA of three warpgroups (384 threads) is launched with 168
// registers a thread, all that a one-CTA SM has (launch bounds 384, 1). The
// warpgroup of the producer and the issuer gives up 96 of them, each of the two
// compute warpgroups takes 48 more: 72 + 2 * 216 = 3 * 168, so the split fits
// the CTA's own allotment and no increase can wait for registers that never
// come. diff_kernel_ready makes sure of the 168 before the first launch.
constexpr int kDiffThreads = 384, kDiffLaunchRegs = 168;
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
// Checked and set once per kernel and device (the calls cost several us).
// done: one bit per device, of one kernel.
inline cudaError_t diff_kernel_ready(std::atomic<unsigned long long>& done, const void* kern, int smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load() >> dev & 1)) return cudaSuccess;
  cudaFuncAttributes a;
  if ((e = cudaFuncGetAttributes(&a, kern)) != cudaSuccess) return e;
  if (a.numRegs != kDiffLaunchRegs) return cudaErrorInvalidConfiguration;
  if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
  if (dev < 64) done.fetch_or(1ull << dev);
  return cudaSuccess;
}

// Programmatic launch: the kernels of one pass follow each other closely (each
// may be put on the GPU while the one before runs out). Every kernel of the
// chain begins with pdl_start: it waits until the one before is done and its
// writes are visible, before it touches memory. The first of a pass is launched
// the ordinary way, behind everything in the stream.
__device__ __forceinline__ void pdl_start() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_next(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&c, kern, args...);
}

// The tile of a CTA, asked for at the start and looked at behind the CTA's set-up.
struct TileLoad {
  int4 used, t;
  int b;                      // its sequence
  __device__ __forceinline__ void ask(const DiffTile* tiles, const int* seq, const DiffGeom& g, int rank) {
    const int4 *pu = tiles + g.ntile, *pt = tiles + rank;
    const int* ps = seq + rank;
    asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(used.x), "=r"(used.y), "=r"(used.z), "=r"(used.w) : "l"(pu));
    asm volatile("ld.global.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(t.x), "=r"(t.y), "=r"(t.z), "=r"(t.w) : "l"(pt));
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(b) : "l"(ps));
  }
  // The entry is in use (like diff_used).
  __device__ __forceinline__ bool live(const DiffGeom& g, int rank, int* err) const {
    if (used.y == g.tag) return rank < used.x;
    if (threadIdx.x == 0) report_error(err, LH_ERR_DEVICE, 404);
    return false;
  }
};
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Results leave through shared memory: a thread holds a row (its TMEM lane), and
// 32 rows' 16-byte pieces stored from there would be 32 lines to an instruction,
// half of each sector. A warp puts its 32 rows of CH pieces into a swizzled buffer
// of its own and stores whole runs of a row. With the tile asked for ahead of the
// set-up: sequences of 512 tokens, 592 tiles x 4 heads of 128, forward 281 -> 199 us,
// dk/dv 268 -> 231, dq 210 -> 197; 16 heads of 8,192 tokens 424 -> 403, 658 -> 652,
// 502 -> 491.
__device__ __forceinline__ uint32_t piece_at(int x) { return (uint32_t)((x & ~7) | ((x ^ (x >> 3)) & 7)) * 16; }
template <int CH>
__device__ __forceinline__ void put_piece(uint8_t* buf, int lane, int c, const uint4& v) {
  *reinterpret_cast<uint4*>(buf + piece_at(lane * CH + c)) = v;
}
// rows: how many of the warp's rows there are
template <int CH, typename T>
__device__ __forceinline__ void put_rows(const uint8_t* buf, int lane, T* dst, long long ld, int rows) {
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int x = i * 32 + lane, r = x / CH, c = x % CH;
    if (r < rows) *reinterpret_cast<uint4*>(dst + r * ld + 8 * c) = *reinterpret_cast<const uint4*>(buf + piece_at(x));
  }
}

// 16-wide slice i of a K-major tile's rows, as an offset of its descriptor
__device__ __forceinline__ uint64_t kslice(int i) {
  return (uint64_t)((i >> 2) * (kDSub >> 4) + (i & 3) * 2);
}

bool make_tmap_16(CUtensorMap* m, const void* base, int D, int S, int BH, bool fp16, int box_rows);

cudaError_t launch_diff_fwd_tc(const DiffGeom& g, const DiffTC& b, const void* q, const void* k, const void* v,
                               const void* lam, void* o, int train, int* err, cudaStream_t s);
cudaError_t launch_diff_bwd_tc(const DiffGeom& g, const DiffTC& b, const void* dout, const void* lam, void* dq, void* dk,
                               void* dv, void* dlam, int* err, cudaStream_t s);

}  // namespace lh
