// Causal differential attention on the tensor cores, backward pass (fp16
// operands, fp32 accumulate, deterministic: no atomics on results).
//
// With A_m recomputed from the forward's row statistics:
//   dv = (A1 - lam A2)^T do,  dP = do v^T (one product, both maps read it),
//   dS1 = A1 (dP - d1),  dS2 = -lam A2 (dP - d2),  d_m = <do, A_m v>,
//   dq_m = dS_m k_m / sqrt(D/2),  dk_m = dS_m^T q_m / sqrt(D/2),  dlam = -sum d2.
// A query that sees one key has A = 1 and dS = 0 exactly; its dS is set to zero
// rather than left to the rounding of dP - d.
//
// Ranges. Gradients of one sequence differ by many powers of two from row to row,
// so every row of do is copied times a power of its own, 2^-e, which leaves the
// row's products as a factor. The maps are held at 2^sp (1 + |lam| below
// 2^(14 - sp)), dS at 2^sh from the bound |dP - d| <= 2 |do row|_1 max |v|:
// no dS leaves fp16 whatever the data.
// - dq: a query row is a lane, so sh and e are the row's own: a dS is normal
//   down to 2^-29 of that bound, and neither another row's do nor its place in the
//   sequence matters.
// - dk, dv: the rows of all queries that see a key tile enter one sum. E is the
//   largest e of that walk and sh from its largest row; A enters times
//   2^(sp + e - E), so that A dos and A (dP - d) come out at one power. What a row
//   adds there keeps its bits down to 2^-29 of the walk's bound (dk) and to 2^-27
//   of its largest do (dv); below, it is off by 2^-40 and 2^-38 of them at most.
//   The keys that only small rows see are another walk with its own E.
// (With one power per sequence and head, from 2 D max |v| max |do|, rows whose do was
// 2^-14 of the largest were off by 1.2 % (dq) and 1.9 % (dk) at 4,096 tokens, by 30
// and 39 % at 8,192 with one v of 100; now 0.17 %, the rounding to bf16, down to 2^-20.)
// The powers are taken out of the fp32 results.
//
// k_diff_pack_do copies do and forms d1, d2 in the same pass, both in the copy's
// units (times 2^-(e + ev)). (The sum of d2 that dlam needs is formed as the sum of
// A2 dP in the dq kernel, from fp32 values: a sum over a long sequence can be small
// beside its terms, and the saved outputs' 11 bits would show in it.)
//
// k_diff_dkdv_tc: one CTA per key tile and key/value head, over the query tiles
// from its own on, of every query head that shares it. Work per pair of tiles:
// X = S_1^T, S_2^T (128 x 128 x D/2 each), Y = dP^T, dV (D), dK_1, dK_2 (D/2
// each): 4 products of 128^3 for D = 128, none twice. TMEM holds X, Y, dV and dK
// (128 columns each, all 512), so X serves the two maps in turn and Y's
// columns, once dP is in registers, take the operands: each 32-column chunk
// holds dS_1 (then dS_2, once dK_1 has read it) in its first 16 and A1 (then A1 -
// lam A2) in its last 16. Order of the products:
//   X_2(t), dK_1(t), X_1(t+1), dV(t), dK_2(t), Y(t+1)
// A warp of its own brings the queries' statistics, three tiles ahead.
// k_diff_dq_tc: one CTA per query tile and head, over the key tiles up to its
// own: X_1, X_2, Y, dQ_1, dQ_2, TMEM X_1 | X_2 | Y | dQ. Both scores of tile t+1
// run under the exponentials of tile t, dQ(t) and Y(t+1) under those of t+1.
// 32,768 exponentials per pair in each kernel: 2,048 cycles of the special-
// function unit against 2,048 (dk, dv) and 1,536 (dq) tensor cycles. Measured at 16
// heads of 8,192 tokens, D = 128: 630 and 458 us (696 and 512 in a long loop under the
// power cap), 5,100 and 3,300 cycles per pair:
// the two warpgroups exponentiate (1,050 cycles per map) and multiply (470 .. 700)
// at the same time, so the two pipes take turns. Giving each warpgroup its own
// 64-column halves, half a tile apart, was slower (1,000 and 800 us): score products
// of N = 64 and twice as many of them.
#include "k_diff_tc.cuh"

namespace lh {
namespace {

using namespace tc;

constexpr int kStages = 3;
constexpr int kComputeWarps = 8;
constexpr uint32_t kX = 0, kY = 128, kAcc0 = 256, kAcc1 = 384;   // dkdv: X, Y, dV, dK
constexpr uint32_t kQX2 = 128, kQY = 256, kQAcc = 384;           // dq: X_1 at 0, X_2, Y, dQ

// NA: stages of A_t (scores and last product). Two serve the dk, dv kernel (its
// scores of tile t + 1 come in the middle of tile t), which needs the room for
// the statistics; the dq kernel, whose scores come first, has three.
constexpr int kVecStages = 3, kVecFloats = 4 * 128 + 4;
template <int D, int NA>
struct BwdLayout {
  static constexpr int SUB = D / 64;
  static constexpr int OPB = SUB * kDSub;
  static constexpr int NSTA = NA, NSTB = 2;         // stages of A_t, B_t
  static constexpr int FIX0 = 0, FIX1 = OPB, RA = 2 * OPB, RB = RA + NSTA * OPB;
  static constexpr int TILES = RB + NSTB * OPB;
  // barriers, the queries' statistics (NA = 2), up to the next 1,024-byte
  // boundary. With three stages of D = 128 that leaves 1,024 bytes of a CTA's shared
  // memory: the base is not aligned here but has to be (base_ok checks it).
  static constexpr int VEC = 256;
  static constexpr int HEAD = NA == 2 ? 7168 : 2048;
  // the walk's WalkScale (NA = 2), or a float4 of each compute warp's factors and
  // behind them 2^e of each compute thread's row (NA = 3)
  static constexpr int FAC = NA == 2 ? HEAD - 64 : 1024 - kComputeWarps * 16;
  static constexpr int BYTES = HEAD + TILES;
  static_assert(NA != 2 || 64 + VEC + kVecStages * kVecFloats * 4 <= HEAD, "statistics");
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct BwdBars {
  uint64_t fix_full, ring_full[kStages][2], ring_empty[kStages][2];
  uint64_t x_full[2], x_free[2], y_full, ds1_ready, dk1_done, p_ready, ds_ready, done, drain;
  uint64_t vec_full[kVecStages], vec_empty[kVecStages];
  uint32_t tmem_base;
  Abort abort;
};
static_assert(sizeof(BwdBars) <= 256, "barrier block");

// Powers of two of one sequence and key/value head.
struct Powers {
  int eq, ek, ev, sp;
  int vx;                     // the v copy is below 2^vx
  int ll;                     // |lam| <= 2^ll, ll >= 0
};
__device__ __forceinline__ Powers powers(const DiffGeom& g, const uint32_t* amax, const __nv_bfloat16* lam, int b, int hk) {
  const size_t plane = (size_t)g.B * g.Hk, at = (size_t)b * g.Hk + hk;
  const uint32_t av = amax[kScaleV * plane + at];
  Powers p;
  p.eq = diff_exp(amax[kScaleQ * plane + at]);
  p.ek = diff_exp(amax[kScaleK * plane + at]);
  p.ev = diff_exp(av);
  p.vx = (int)(av >> 23) - 126 - p.ev;
  float lm = 0.f;
  for (int h = hk * g.G; h < (hk + 1) * g.G; ++h) lm = fmaxf(lm, fabsf(__bfloat162float(lam[h])));
  lm = fminf(lm, 1e30f);
  p.sp = max(-100, 13 - ilogbf(1.f + lm));
  p.ll = lm > 1.f ? ilogbf(lm) + 1 : 0;
  return p;
}
// What a walk of dk, dv is scaled by: f = 2^(sh - sp), the scores' 2^(eq + ek), the
// results' factors; sp - E.
struct WalkScale {
  float f, s, dv, dk;
  int base;
};
// 2^sh for dS of rows (of the do copy) with a 1-norm below 2^xn: |dS| 2^sh < 2^15
__device__ __forceinline__ int ds_exp(const Powers& p, int xn, int ll) { return max(-60, min(24, 14 - xn - p.vx - ll)); }

// The largest e and the largest exponent of a row's 1-norm over the query tiles of a
// walk (padded tiles first .. first + per - 1 of the group's heads); a whole warp.
__device__ __forceinline__ void walk_max(const int* tmax, const DiffGeom& g, int hk, int first, int per, int& E, int& X) {
  E = X = -32768;
  for (int h = hk * g.G; h < (hk + 1) * g.G; ++h)
    for (int i = threadIdx.x & 31; i < per; i += 32) {
      const int w = tmax[(size_t)h * g.ntile + first + i];
      E = max(E, row_e(w));
      X = max(X, row_x(w));
    }
  E = max(__reduce_max_sync(0xffffffffu, E), -kScaleMaxExp);      // rows of zeros alone
  X = __reduce_max_sync(0xffffffffu, X);
}

// The swizzled tiles need a 1,024-byte aligned base; dynamic shared memory starts
// at one (declared so, and checked before anything is written).
__device__ __forceinline__ bool base_ok(const void* raw, int* err) {
  if ((smem_u32(raw) & 1023u) == 0) return true;
  if (threadIdx.x == 0) report_error(err, LH_ERR_DEVICE, 403);
  return false;
}

__device__ __forceinline__ void bwd_setup(BwdBars* bars, int warp) {
  if (threadIdx.x == 0) {
    mbar_init(&bars->fix_full, 1);
    for (int s = 0; s < kStages; ++s)
      for (int o = 0; o < 2; ++o) {
        mbar_init(&bars->ring_full[s][o], 1);
        mbar_init(&bars->ring_empty[s][o], 1);
      }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->x_full[s], 1);
      mbar_init(&bars->x_free[s], kComputeWarps);
    }
    for (int s = 0; s < kVecStages; ++s) {
      mbar_init(&bars->vec_full[s], 1);
      mbar_init(&bars->vec_empty[s], kComputeWarps);
    }
    mbar_init(&bars->y_full, 1);
    mbar_init(&bars->ds1_ready, kComputeWarps);
    mbar_init(&bars->dk1_done, 1);
    mbar_init(&bars->p_ready, kComputeWarps);
    mbar_init(&bars->ds_ready, kComputeWarps);
    mbar_init(&bars->done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort.flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

__device__ __forceinline__ void bwd_teardown(uint32_t tbase, int warp) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// The two fixed tiles (rows frow .. of head fh), then n streamed tiles: step t
// reads rows row0 + (t % per) * 128 of head h0 + t / per.
template <typename Lay>
__device__ void bwd_produce(uint8_t* sm, BwdBars* bars, const CUtensorMap* f0, const CUtensorMap* f1, int frow, int fh,
                            const CUtensorMap* ma, const CUtensorMap* mb, int row0, int per, int h0, int n,
                            volatile Abort* ab, int* err) {
  constexpr int SUB = Lay::SUB, NSTA = Lay::NSTA, NSTB = Lay::NSTB;
  mbar_expect_tx(&bars->fix_full, 2 * Lay::OPB);
  for (int c = 0; c < SUB; ++c) {
    tma_load_3d(sm + Lay::FIX0 + c * kDSub, f0, &bars->fix_full, 64 * c, frow, fh);
    tma_load_3d(sm + Lay::FIX1 + c * kDSub, f1, &bars->fix_full, 64 * c, frow, fh);
  }
  int issued = 0, i = 0, h = h0;
  for (int t = 0; t < n; ++t) {
    bool go = true;
    for (int o = 0; o < 2; ++o) {
      const int nst = o ? NSTB : NSTA, st = t % nst;
      if (t >= nst && !mbar_wait(&bars->ring_empty[st][o], ((t / nst) - 1) & 1, ab, err, 41)) {
        go = false;
        break;
      }
      uint64_t* full = &bars->ring_full[st][o];
      uint8_t* dst = sm + (o ? Lay::RB : Lay::RA) + st * Lay::OPB;
      mbar_expect_tx(full, Lay::OPB);
      for (int c = 0; c < SUB; ++c) tma_load_3d(dst + c * kDSub, o ? mb : ma, full, 64 * c, row0 + i * 128, h);
      issued = 2 * t + o + 1;
    }
    if (!go) break;
    if (++i == per) {
      i = 0;
      ++h;
    }
  }
  if (ab->flag) {
    // wind-down: let the copies still in flight land before the CTA exits
    Abort none{0};
    mbar_wait(&bars->fix_full, 0, &none, nullptr, 0);
    const int na = (issued + 1) / 2, nb = issued / 2;
    for (int x = na - NSTA < 0 ? 0 : na - NSTA; x < na; ++x)
      mbar_wait(&bars->ring_full[x % NSTA][0], (x / NSTA) & 1, &none, nullptr, 0);
    for (int x = nb - NSTB < 0 ? 0 : nb - NSTB; x < nb; ++x)
      mbar_wait(&bars->ring_full[x % NSTB][1], (x / NSTB) & 1, &none, nullptr, 0);
  }
}

// Descriptors and waits of the issuing warp (all lanes wait, one issues).
template <int D, typename Lay>
struct Issuer {
  static constexpr uint32_t IDX = idesc_f16(128, 128, false);
  static constexpr uint32_t IDV = idesc_f16(128, D, true), IDM = idesc_f16(128, D / 2, true);
  static constexpr uint32_t OPB16 = Lay::OPB >> 4;
  static constexpr int KS = D / 32;
  // the second map's columns of an MN-major tile: a slab on (D = 128), or 64
  // bytes on within the slab (D = 64)
  static constexpr uint32_t MAP2 = D == 128 ? (kDSub >> 4) : 4;
  uint64_t dF0, dF1, dA, dB, dAm, dBm;
  BwdBars* bars;
  volatile Abort* ab;
  int* err;
  bool leader;

  __device__ Issuer(uint8_t* sm, BwdBars* b, volatile Abort* a, int* e) : bars(b), ab(a), err(e) {
    const uint32_t s = smem_u32(sm);
    dF0 = sdesc_sw128(s + Lay::FIX0, 16, 1024);
    dF1 = sdesc_sw128(s + Lay::FIX1, 16, 1024);
    dA = sdesc_sw128(s + Lay::RA, 16, 1024);
    dB = sdesc_sw128(s + Lay::RB, 16, 1024);
    dAm = sdesc_sw128(s + Lay::RA, kDSub, 1024);
    dBm = sdesc_sw128(s + Lay::RB, kDSub, 1024);
    leader = elect_one();
  }
  __device__ bool wait(uint64_t* bar, uint32_t parity, int site) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, err, site));
  }
  __device__ bool ring(int t, int o) {
    const int nst = o ? Lay::NSTB : Lay::NSTA;
    return wait(&bars->ring_full[t % nst][o], (t / nst) & 1, 43);
  }
  __device__ void score(uint32_t dst, int m, int t, uint64_t* bar) {     // F0_m A_t_m^T
    const uint64_t b0 = dA + (uint64_t)((t % Lay::NSTA) * OPB16);
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) umma_f16(dst, dF0 + kslice(m * KS + kk), b0 + kslice(m * KS + kk), IDX, kk > 0 ? 1u : 0u);
      umma_commit(bar);
    }
  }
  __device__ void dp(uint32_t dst, int t) {                              // F1 B_t^T
    const uint64_t b0 = dB + (uint64_t)((t % Lay::NSTB) * OPB16);
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) umma_f16(dst, dF1 + kslice(kk), b0 + kslice(kk), IDX, kk > 0 ? 1u : 0u);
      umma_commit(&bars->y_full);
    }
  }
  // acc += operand * (columns of map m of A_t); operand slice kk at acol(kk)
  template <typename F>
  __device__ void grad(uint32_t acc, int m, int t, F acol) {
    const uint64_t b0 = dAm + (uint64_t)((t % Lay::NSTA) * OPB16 + (m ? MAP2 : 0u));
    if (leader) {
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) umma_f16_ts(acc, acol(kk), b0 + kk * 128, IDM, (t > 0 || kk > 0) ? 1u : 0u);
    }
  }
  __device__ void commit(uint64_t* bar) {
    if (leader) umma_commit(bar);
  }
  __device__ void finish(bool ok) {
    if (leader) {
      if (ok) umma_commit(&bars->done);
      umma_commit(&bars->drain);
    }
    __syncwarp();
    Abort none{0};
    mbar_wait(&bars->drain, 0, &none, nullptr, 0);
  }
};

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// 32 columns of a key row: A^T 2^sp = 2^(S^T c2 + nl), nl of the columns' queries
// (broadcast reads). MASK: columns before the key's own position get 0.
template <bool MASK>
__device__ __forceinline__ void map_cols(uint32_t (&s)[32], const float* nl, float c2, int col0, int first) {
  const float2 cc = make_float2(c2, c2);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 a = *reinterpret_cast<const float4*>(nl + e);
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      const float2 x = __ffma2_rn(f2(s[e + u], s[e + u + 1]), cc, u ? make_float2(a.z, a.w) : make_float2(a.x, a.y));
      float p0 = ex2(x.x), p1 = ex2(x.y);
      if (MASK) {
        if (col0 + e + u < first) p0 = 0.f;
        if (col0 + e + u + 1 < first) p1 = 0.f;
      }
      s[e + u] = __float_as_uint(p0);
      s[e + u + 1] = __float_as_uint(p1);
    }
  }
}
// dS 2^sh = A (f dP + nd) for 32 columns with the columns' nd, as fp16 pairs
__device__ __forceinline__ void ds_cols(const uint32_t (&p)[32], const uint32_t (&d)[32], const float* nd, float f,
                                        uint32_t (&pk)[16]) {
  const float2 ff = make_float2(f, f);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 b = *reinterpret_cast<const float4*>(nd + e);
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      const float2 x = __ffma2_rn(f2(d[e + u], d[e + u + 1]), ff, u ? make_float2(b.z, b.w) : make_float2(b.x, b.y));
      pk[(e + u) >> 1] = h2_bits(__float22half2_rn(__fmul2_rn(f2(p[e + u], p[e + u + 1]), x)));
    }
  }
}

// ---------------------------------------------------------------- dk, dv
template <int D>
__global__ void __launch_bounds__(kDiffThreads, 1)
k_diff_dkdv_tc(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo, const DiffGeom g,
               const __nv_bfloat16* __restrict__ lam, const DiffTile* __restrict__ tiles, const int* __restrict__ seq,
               const uint32_t* __restrict__ amax, const int* __restrict__ rowx, const int* __restrict__ tmax,
               const float* __restrict__ lse, const float* __restrict__ delta, __nv_bfloat16* __restrict__ dk,
               __nv_bfloat16* __restrict__ dv, float c2, float scale, int* err) {
  using Lay = BwdLayout<D, 2>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem_raw);
  uint8_t* sm = smem_raw + Lay::HEAD;
  int rank, hk;
  diff_place(g.ok, blockIdx.x, rank, hk);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!base_ok(smem_raw, err)) return;                          // the whole CTA
  if (threadIdx.x == 0) {
    prefetch_map(&tk);
    prefetch_map(&tv);
    prefetch_map(&tq);
    prefetch_map(&tdo);
  }
  pdl_start();
  TileLoad ask;
  ask.ask(tiles, seq, g, rank);
  bwd_setup(bars, warp);
  const uint32_t tbase = bars->tmem_base;
  volatile Abort* ab = &bars->abort;
  if (!ask.live(g, rank, err)) {                                // the whole CTA
    if (warp == 1) tmem_dealloc(tbase, 512);
    return;
  }
  const DiffTile tl = tiles[rank];
  const int nt = (tl.y + 127) / 128, j = nt - 1 - tl.w;      // early key tiles first: they have the most queries
  const int per = nt - j, n = per * g.G;                      // query tiles j .. nt - 1 of each head
  WalkScale* ws = reinterpret_cast<WalkScale*>(smem_raw + Lay::FAC);
  if (warp < 4) regs_give();
  if (warp == 0) {
    if (lane == 0)
      bwd_produce<Lay>(sm, bars, &tk, &tv, tl.z + j * 128, hk, &tq, &tdo, tl.z + j * 128, per, hk * g.G, n, ab, err);
  } else if (warp == 1) {
    Issuer<D, Lay> is(sm, bars, ab, err);
    const uint32_t tX = tbase + kX, tY = tbase + kY;
    auto ds_at = [&](int kk) -> uint32_t { return tY + 32 * (kk >> 1) + 8 * (kk & 1); };
    bool ok = is.wait(&bars->fix_full, 0, 42) && is.ring(0, 0);
    if (ok) {
      tc_fence_after();
      is.score(tX, 0, 0, &bars->x_full[0]);
      ok = is.ring(0, 1);
    }
    if (ok) is.dp(tY, 0);
    for (int t = 0; ok && t < n; ++t) {
      const bool more = t + 1 < n;
      ok = is.wait(&bars->x_free[0], t & 1, 44);
      if (!ok) break;
      tc_fence_after();
      is.score(tX, 1, t, &bars->x_full[1]);
      ok = is.wait(&bars->ds1_ready, t & 1, 45);
      if (!ok) break;
      tc_fence_after();
      is.grad(tbase + kAcc1, 0, t, ds_at);
      is.commit(&bars->dk1_done);
      ok = is.wait(&bars->x_free[1], t & 1, 44) && (!more || is.ring(t + 1, 0));
      if (!ok) break;
      if (more) {
        tc_fence_after();
        is.score(tX, 0, t + 1, &bars->x_full[0]);
      }
      ok = is.wait(&bars->p_ready, t & 1, 46);
      if (!ok) break;
      tc_fence_after();
      if (is.leader) {
        const uint64_t b0 = is.dBm + (uint64_t)((t % Lay::NSTB) * Issuer<D, Lay>::OPB16);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_ts(tbase + kAcc0, ds_at(kk) + 16, b0 + kk * 128, Issuer<D, Lay>::IDV, (t > 0 || kk > 0) ? 1u : 0u);
      }
      is.commit(&bars->ring_empty[t % Lay::NSTB][1]);
      ok = is.wait(&bars->ds_ready, t & 1, 47);
      if (!ok) break;
      tc_fence_after();
      is.grad(tbase + kAcc1 + D / 2, 1, t, ds_at);
      is.commit(&bars->ring_empty[t % Lay::NSTA][0]);
      if (more) {
        ok = is.ring(t + 1, 1);
        if (!ok) break;
        is.dp(tY, t + 1);
      }
    }
    is.finish(ok);
  } else if (warp == 3) {
    // the walk's powers of two, for the warps that need them
    const Powers pw = powers(g, amax, lam, seq[rank], hk);
    int E, X;
    walk_max(tmax, g, hk, (tl.z >> 7) + j, per, E, X);
    const int sh = ds_exp(pw, X - E, pw.ll);
    if (lane == 0) {
      ws->f = pow2f(sh - pw.sp);
      ws->s = pow2f(pw.eq + pw.ek);
      ws->dv = pow2f(E) * pow2f(-pw.sp);
      ws->dk = scale * pow2f(E + pw.ev) * pow2f(pw.eq - sh);
      ws->base = pw.sp - E;
    }
    named_bar_sync(1, 320);              // warps 2 .. 11
  } else if (warp == 2) {
    named_bar_sync(1, 320);
    // the queries' statistics, a few tiles ahead of the compute warps: [0] -lse 1,
    // [1] -lse 2 + log2 |lam| (both + sp + e - E), [2] -d1, [3] -d2 in dS units and
    // signed like the map in A1 - lam A2; then that sign. Rows past the end: zeros,
    // so that dS = 0 there.
    const size_t rows = (size_t)g.ntile * 128;
    const float md = -ws->f;
    const int base = ws->base;
    int i = j, h = hk * g.G;
    for (int t = 0; t < n; ++t) {
      const int st = t % kVecStages;
      if (t >= kVecStages &&
          !__all_sync(0xffffffffu, mbar_wait(&bars->vec_empty[st], ((t / kVecStages) - 1) & 1, ab, err, 52)))
        break;
      float* vec = reinterpret_cast<float*>(smem_raw + Lay::VEC) + st * kVecFloats;
      const float l = __bfloat162float(lam[h]), sg = l > 0.f ? -1.f : 1.f, ll = log2f(fabsf(l));
      const int q = i * 128 + 4 * lane;
      const int4 w = *reinterpret_cast<const int4*>(rowx + (size_t)h * rows + tl.z + q);
      const float4 ad = make_float4((float)(base + row_e(w.x)), (float)(base + row_e(w.y)), (float)(base + row_e(w.z)),
                                    (float)(base + row_e(w.w)));
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int mp = v & 1;
        const float4 x = *reinterpret_cast<const float4*>((v < 2 ? lse : delta) + ((size_t)h * 2 + mp) * rows + tl.z + q);
        const float add = mp ? ll : 0.f, mul = md * (mp ? sg : 1.f);
        float4 y;
        y.x = q < tl.y ? (v < 2 ? ad.x + add - x.x : x.x * mul) : 0.f;
        y.y = q + 1 < tl.y ? (v < 2 ? ad.y + add - x.y : x.y * mul) : 0.f;
        y.z = q + 2 < tl.y ? (v < 2 ? ad.z + add - x.z : x.z * mul) : 0.f;
        y.w = q + 3 < tl.y ? (v < 2 ? ad.w + add - x.w : x.w * mul) : 0.f;
        *reinterpret_cast<float4*>(vec + 128 * v + 4 * lane) = y;
      }
      if (lane == 0) vec[512] = sg;
      mbar_arrive_warp(&bars->vec_full[st]);
      if (++i == nt) {
        i = j;
        ++h;
      }
    }
  } else if (warp >= 4) {
    regs_take();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;                   // which 64 of the 128 columns
    const int m = quarter * 32 + lane;                  // key row within the tile / TMEM lane
    const uint32_t la = (uint32_t)(quarter * 32) << 16;
    const uint32_t cX = tbase + la + kX + 64 * half, cY = tbase + la + kY + 64 * half;
    named_bar_sync(1, 320);
    const float f = ws->f;
    c2 *= ws->s;
    bool ok = true;
    int i = j;
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, err, site));
    };
    for (int t = 0; t < n; ++t) {
      const bool diag = i == j;
      const bool zero = diag && i == 0 && half == 0;    // column 0 is the sequence's first query: dS = 0
      const float* vec = reinterpret_cast<const float*>(smem_raw + Lay::VEC) + (t % kVecStages) * kVecFloats + 64 * half;
      ok = wait(&bars->vec_full[t % kVecStages], (t / kVecStages) & 1, 53) && wait(&bars->x_full[0], t & 1, 48);
      if (!ok) break;
      tc_fence_after();
      uint32_t p0[32], p1[32], d0[32], d1[32], pk[16];
      tmem_ld32(cX, p0);
      tmem_ld32(cX + 32, p1);
      tmem_wait_ld_regs(p0);
      reg_fence32(p1);
      tc_fence_before();
      mbar_arrive_warp(&bars->x_free[0]);
      if (diag) {
        map_cols<true>(p0, vec, c2, 64 * half, m);
        map_cols<true>(p1, vec + 32, c2, 64 * half + 32, m);
      } else {
        map_cols<false>(p0, vec, c2, 0, 0);
        map_cols<false>(p1, vec + 32, c2, 0, 0);
      }
      ok = wait(&bars->y_full, t & 1, 49);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(cY, d0);
      tmem_ld32(cY + 32, d1);
      tmem_wait_ld_regs(d0);
      reg_fence32(d1);
      ds_cols(p0, d0, vec + 256, f, pk);
      if (zero) pk[0] &= 0xFFFF0000u;
      tmem_st16(cY, pk);
      ds_cols(p1, d1, vec + 288, f, pk);
      tmem_st16(cY + 32, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(&bars->ds1_ready);
      // A1 waits as fp16 pairs in the columns of A1 - lam A2 (fp32 would take 32
      // more registers; its rounding, 2^-12 of A1, is half of the sum's own)
      uint32_t a0[16], a1[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        a0[e] = pack_f16(__uint_as_float(p0[2 * e]), __uint_as_float(p0[2 * e + 1]));
        a1[e] = pack_f16(__uint_as_float(p1[2 * e]), __uint_as_float(p1[2 * e + 1]));
      }
      ok = wait(&bars->x_full[1], t & 1, 48);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(cX, p0);
      tmem_ld32(cX + 32, p1);
      tmem_wait_ld_regs(p0);
      reg_fence32(p1);
      tc_fence_before();
      mbar_arrive_warp(&bars->x_free[1]);
      if (diag) {
        map_cols<true>(p0, vec + 128, c2, 64 * half, m);
        map_cols<true>(p1, vec + 160, c2, 64 * half + 32, m);
      } else {
        map_cols<false>(p0, vec + 128, c2, 0, 0);
        map_cols<false>(p1, vec + 160, c2, 0, 0);
      }
      // p: |lam| A2; A1 - lam A2 into its columns
      const float s2 = vec[512 - 64 * half];
      const float2 sg2 = make_float2(s2, s2);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        a0[e] = h2_bits(__float22half2_rn(
            __ffma2_rn(f2(p0[2 * e], p0[2 * e + 1]), sg2, __half22float2(*reinterpret_cast<const __half2*>(&a0[e])))));
        a1[e] = h2_bits(__float22half2_rn(
            __ffma2_rn(f2(p1[2 * e], p1[2 * e + 1]), sg2, __half22float2(*reinterpret_cast<const __half2*>(&a1[e])))));
      }
      tmem_st16(cY + 16, a0);
      tmem_st16(cY + 48, a1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(&bars->p_ready);
      ds_cols(p0, d0, vec + 384, f * s2, a0);
      if (zero) a0[0] &= 0xFFFF0000u;
      ds_cols(p1, d1, vec + 416, f * s2, a1);
      mbar_arrive_warp(&bars->vec_empty[t % kVecStages]);
      ok = wait(&bars->dk1_done, t & 1, 50);
      if (!ok) break;
      tc_fence_after();
      tmem_st16(cY, a0);
      tmem_st16(cY + 32, a1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(&bars->ds_ready);
      if (++i == nt) i = j;
    }
    if (ok && __all_sync(0xffffffffu, mbar_wait(&bars->done, 0, ab, err, 51))) {
      tc_fence_after();
      const int key = j * 128 + m;
      const float mv = ws->dv, mk = ws->dk;
      constexpr int CH = D / 16, BUF = 32 * CH * 16;
      uint8_t* buf = sm + (warp - 4) * 2 * BUF;           // the operands' memory: all products are done
#pragma unroll 1
      for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
        // warp-collective loads: every lane runs them
        uint32_t a[32], b[32];
        tmem_ld32(tbase + la + kAcc0 + 32 * c, a);
        tmem_ld32(tbase + la + kAcc1 + 32 * c, b);
        tmem_wait_ld_regs(a);
        reg_fence32(b);
        bool fin = true;
#pragma unroll
        for (int e = 0; e < 32; ++e) fin &= fabsf(__uint_as_float(b[e])) < INFINITY;
        if (!fin && key < tl.y) report_error(err, LH_ERR_DEVICE, 101);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 u, w;
          uint32_t *pu = &u.x, *pw4 = &w.x;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            pu[x] = pack_bf16(__uint_as_float(a[e + 2 * x]) * mv, __uint_as_float(a[e + 2 * x + 1]) * mv);
            pw4[x] = pack_bf16(__uint_as_float(b[e + 2 * x]) * mk, __uint_as_float(b[e + 2 * x + 1]) * mk);
          }
          const int piece = 4 * (c - half * (D / 64)) + e / 8;
          put_piece<CH>(buf, lane, piece, u);
          put_piece<CH>(buf + BUF, lane, piece, w);
        }
      }
      __syncwarp();
      const int first = j * 128 + quarter * 32, live = tl.y - first;
      const long long col = (long long)hk * D + half * (D / 2);
      put_rows<CH>(buf, lane, dv + (long long)(tl.x + first) * g.ldv + col, g.ldv, live);
      put_rows<CH>(buf + BUF, lane, dk + (long long)(tl.x + first) * g.ldk + col, g.ldk, live);
    }
  }
  bwd_teardown(tbase, warp);
}

// ---------------------------------------------------------------- dq
// 64 columns of a query row: A 2^sp = 2^(S c2 + nl). MASK: key columns past `last` get 0.
template <bool MASK>
__device__ __forceinline__ void map_row(uint32_t (&s)[32], float nl, float c2, int col0, int last) {
  const float2 cc = make_float2(c2, c2), nn = make_float2(nl, nl);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 x = __ffma2_rn(f2(s[e], s[e + 1]), cc, nn);
    float p0 = ex2(x.x), p1 = ex2(x.y);
    if (MASK) {
      if (col0 + e > last) p0 = 0.f;
      if (col0 + e + 1 > last) p1 = 0.f;
    }
    s[e] = __float_as_uint(p0);
    s[e + 1] = __float_as_uint(p1);
  }
}

template <int D>
__global__ void __launch_bounds__(kDiffThreads, 1)
k_diff_dq_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
             const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const DiffGeom g,
             const __nv_bfloat16* __restrict__ lam, const DiffTile* __restrict__ tiles, const int* __restrict__ seq,
             const uint32_t* __restrict__ amax, const int* __restrict__ rowx, const float* __restrict__ lse,
             const float* __restrict__ delta, __nv_bfloat16* __restrict__ dq, float* __restrict__ part, float c2, float scale,
             int* err) {
  using Lay = BwdLayout<D, 3>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem_raw);
  uint8_t* sm = smem_raw + Lay::HEAD;
  float* red = reinterpret_cast<float*>(smem_raw + 256);          // the compute warps' sums of A2 dP
  int rank, h;
  diff_place(g.oq, blockIdx.x, rank, h);
  const int hk = h / g.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!base_ok(smem_raw, err)) return;                          // the whole CTA
  if (threadIdx.x == 0) {
    prefetch_map(&tq);
    prefetch_map(&tdo);
    prefetch_map(&tk);
    prefetch_map(&tv);
  }
  pdl_start();
  TileLoad ask;
  ask.ask(tiles, seq, g, rank);
  bwd_setup(bars, warp);
  const uint32_t tbase = bars->tmem_base;
  volatile Abort* ab = &bars->abort;
  if (!ask.live(g, rank, err)) {                                // the whole CTA
    if (warp == 1) tmem_dealloc(tbase, 512);
    if (threadIdx.x == 0) part[(size_t)h * g.ntile + rank] = 0.f;
    return;
  }
  const DiffTile tl = tiles[rank];
  const int n = tl.w + 1;
  if (warp < 4) regs_give();
  if (warp == 0) {
    if (lane == 0) bwd_produce<Lay>(sm, bars, &tq, &tdo, tl.z + tl.w * 128, h, &tk, &tv, tl.z, n, hk, n, ab, err);
  } else if (warp == 1) {
    Issuer<D, Lay> is(sm, bars, ab, err);
    // the fixed tiles belong to head h, the streamed ones to hk; operands of
    // slice kk: dS_1 at 16 kk, dS_2 behind it at 16 kk + 8
    auto ds1_at = [&](int kk) -> uint32_t { return tbase + kQY + 16 * kk; };
    auto ds2_at = [&](int kk) -> uint32_t { return tbase + kQY + 16 * kk + 8; };
    bool ok = is.wait(&bars->fix_full, 0, 42) && is.ring(0, 0);
    if (ok) {
      tc_fence_after();
      is.score(tbase, 0, 0, &bars->x_full[0]);
      is.score(tbase + kQX2, 1, 0, &bars->x_full[1]);
      ok = is.ring(0, 1);
    }
    if (ok) {
      is.dp(tbase + kQY, 0);
      is.commit(&bars->ring_empty[0][1]);
    }
    for (int t = 0; ok && t < n; ++t) {
      const bool more = t + 1 < n;
      if (more) {
        ok = is.ring(t + 1, 0) && is.wait(&bars->x_free[0], t & 1, 44);
        if (!ok) break;
        tc_fence_after();
        is.score(tbase, 0, t + 1, &bars->x_full[0]);
        ok = is.wait(&bars->x_free[1], t & 1, 44);
        if (!ok) break;
        tc_fence_after();
        is.score(tbase + kQX2, 1, t + 1, &bars->x_full[1]);
      }
      ok = is.wait(&bars->ds_ready, t & 1, 47);
      if (!ok) break;
      tc_fence_after();
      is.grad(tbase + kQAcc, 0, t, ds1_at);
      is.grad(tbase + kQAcc + D / 2, 1, t, ds2_at);
      is.commit(&bars->ring_empty[t % Lay::NSTA][0]);
      if (more) {
        ok = is.ring(t + 1, 1);
        if (!ok) break;
        is.dp(tbase + kQY, t + 1);
        is.commit(&bars->ring_empty[(t + 1) % Lay::NSTB][1]);
      }
    }
    is.finish(ok);
  } else if (warp >= 4) {
    regs_take();
    const int quarter = warp & 3;
    const int half = (warp - 4) >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t la = (uint32_t)(quarter * 32) << 16;
    const uint32_t cX = tbase + la + 64 * half;
    const int row = tl.w * 128 + r;
    const size_t rows = (size_t)g.ntile * 128, at = (size_t)h * 2 * rows + tl.z + row;
    const bool in = row < tl.y;
    const Powers pw = powers(g, amax, lam, seq[rank], hk);
    const int rw = in ? rowx[(size_t)h * rows + tl.z + row] : 0;
    // the first query of a sequence sees one key: f = d = 0 make its dS zero
    const float f = row > 0 ? pow2f(ds_exp(pw, row_x(rw) - row_e(rw), 0) - pw.sp) : 0.f, md = -f;
    const float nl1 = in ? (float)pw.sp - lse[at] : 0.f, nl2 = in ? (float)pw.sp - lse[at + rows] : 0.f;
    const float nd1 = in ? delta[at] * md : 0.f, nd2 = in ? delta[at + rows] * md : 0.f;
    c2 *= pow2f(pw.eq + pw.ek);
    // what the results are multiplied by waits in shared memory, not in registers
    float4* fac = reinterpret_cast<float4*>(smem_raw + Lay::FAC) + (warp - 4);
    reinterpret_cast<float*>(smem_raw + 1024)[threadIdx.x - 128] = pow2f(row_e(rw));
    if (lane == 0)
      *fac = make_float4(pow2f(pw.ev), pow2f(-pw.sp),
                         scale * pow2f(pw.ev) * pow2f(pw.ek) * (half ? -__bfloat162float(lam[h]) : 1.f), 0.f);
    __syncwarp();
    float2 dl = make_float2(0.f, 0.f);                    // sum of A2 dP of this thread's columns
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      uint32_t a0[32], a1[32], b0[32], b1[32];
      const bool diag = t == tl.w;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->x_full[0], t & 1, ab, err, 48))) { ok = false; break; }
      tc_fence_after();
      tmem_ld32(cX, a0);
      tmem_ld32(cX + 32, a1);
      tmem_wait_ld_regs(a0);
      reg_fence32(a1);
      tc_fence_before();
      mbar_arrive_warp(&bars->x_free[0]);
      if (diag) {
        map_row<true>(a0, nl1, c2, 64 * half, r);
        map_row<true>(a1, nl1, c2, 64 * half + 32, r);
      } else {
        map_row<false>(a0, nl1, c2, 0, 0);
        map_row<false>(a1, nl1, c2, 0, 0);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->x_full[1], t & 1, ab, err, 48))) { ok = false; break; }
      tc_fence_after();
      tmem_ld32(cX + kQX2, b0);
      tmem_ld32(cX + kQX2 + 32, b1);
      tmem_wait_ld_regs(b0);
      reg_fence32(b1);
      tc_fence_before();
      mbar_arrive_warp(&bars->x_free[1]);
      if (diag) {
        map_row<true>(b0, nl2, c2, 64 * half, r);
        map_row<true>(b1, nl2, c2, 64 * half + 32, r);
      } else {
        map_row<false>(b0, nl2, c2, 0, 0);
        map_row<false>(b1, nl2, c2, 0, 0);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->y_full, t & 1, ab, err, 49))) { ok = false; break; }
      tc_fence_after();
      const uint32_t cY = cX + kQY;
      const float2 ff = make_float2(f, f), v1 = make_float2(nd1, nd1), v2 = make_float2(nd2, nd2);
      // 16 columns of dP, then both maps' dS (8 packed columns each) into them
      auto cols16 = [&](const uint32_t (&a)[32], const uint32_t (&b)[32], int o, uint32_t at16) {
        uint32_t d[16], pk[16];
        tmem_ld16(at16, d);
        tmem_wait_ld_regs16(d);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 dd = f2(d[e], d[e + 1]);
          dl = __ffma2_rn(f2(b[o + e], b[o + e + 1]), dd, dl);
          pk[e >> 1] = h2_bits(__float22half2_rn(__fmul2_rn(f2(a[o + e], a[o + e + 1]), __ffma2_rn(dd, ff, v1))));
          pk[8 + (e >> 1)] = h2_bits(__float22half2_rn(__fmul2_rn(f2(b[o + e], b[o + e + 1]), __ffma2_rn(dd, ff, v2))));
        }
        tmem_st16(at16, pk);
      };
      cols16(a0, b0, 0, cY);
      cols16(a0, b0, 16, cY + 16);
      cols16(a1, b1, 0, cY + 32);
      cols16(a1, b1, 16, cY + 48);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(&bars->ds_ready);
    }
    const float pe = reinterpret_cast<const float*>(smem_raw + 1024)[threadIdx.x - 128];
    float d2 = (dl.x + dl.y) * fac->x * pe * fac->y;
#pragma unroll
    for (int o = 16; o; o >>= 1) d2 += __shfl_xor_sync(0xffffffffu, d2, o);
    if (lane == 0) red[warp - 4] = d2;
    if (ok && __all_sync(0xffffffffu, mbar_wait(&bars->done, 0, ab, err, 51))) {
      tc_fence_after();
      // dS_2 goes without its factor -lam until here (half 1 holds map 2's columns)
      // 2^-sh = 2^-sp / f, a power of two
      const float mq = f > 0.f ? fac->z * pe * (__int_as_float(0x7F000000 - __float_as_int(f)) * fac->y) : 0.f;
      constexpr int CH = D / 16;
      uint8_t* buf = sm + (warp - 4) * 32 * CH * 16;      // the operands' memory: all products are done
#pragma unroll 1
      for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
        uint32_t a[32];
        tmem_ld32(tbase + la + kQAcc + 32 * c, a);
        tmem_wait_ld_regs(a);
        bool fin = true;
#pragma unroll
        for (int e = 0; e < 32; ++e) fin &= fabsf(__uint_as_float(a[e])) < INFINITY;
        if (!fin && in) report_error(err, LH_ERR_DEVICE, 101);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 u;
          uint32_t* pu = &u.x;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            pu[x] = pack_bf16(__uint_as_float(a[e + 2 * x]) * mq, __uint_as_float(a[e + 2 * x + 1]) * mq);
          put_piece<CH>(buf, lane, 4 * (c - half * (D / 64)) + e / 8, u);
        }
      }
      __syncwarp();
      const int first = tl.w * 128 + quarter * 32;
      put_rows<CH>(buf, lane, dq + (long long)(tl.x + first) * g.ldq + (long long)h * D + half * (D / 2), g.ldq, tl.y - first);
    }
  }
  bwd_teardown(tbase, warp);
  if (threadIdx.x == 0) {
    float d2 = 0.f;
    for (int w = 0; w < kComputeWarps; ++w) d2 += red[w];
    part[(size_t)h * g.ntile + rank] = d2;
  }
}

// ---------------------------------------------------------------- do: working copy, d1, d2
// One 128-row tile of one head; D / 8 lanes to a row.
template <int D>
__global__ void __launch_bounds__(256) k_diff_pack_do(const DiffGeom g, const __nv_bfloat16* __restrict__ dout,
                                                      const __half* __restrict__ om, const DiffTile* __restrict__ tiles,
                                                      __half* __restrict__ dos, float* __restrict__ delta,
                                                      int* __restrict__ rowx, int* __restrict__ tmax, int* err) {
  constexpr int L = D / 8, RPB = 256 / L;      // lanes per row, rows per step
  __shared__ int red[2][8];
  const int h = blockIdx.y, lane = threadIdx.x & 31;
  pdl_start();
  if ((int)blockIdx.x >= diff_used(tiles, g, err)) return;
  const DiffTile t = tiles[blockIdx.x];
  const int r0 = t.w * 128, c = (threadIdx.x % L) * 8;
  const size_t rows = (size_t)g.ntile * 128;
  int E = kRowNone, X = kRowNone;
  bool fin = true;
#pragma unroll 2
  for (int r = threadIdx.x / L; r < 128; r += RPB) {
    const bool in = r0 + r < t.y;
    const size_t prow = (size_t)t.z + r0 + r;
    uint4 raw = make_uint4(0, 0, 0, 0);
    float u[8] = {}, w[8] = {};
    if (in) {
      raw = __ldg(reinterpret_cast<const uint4*>(dout + (long long)(t.x + r0 + r) * g.ldo + (long long)h * D + c));
      Vec8<__half>::load_f32(om + ((size_t)h * 2 * rows + prow) * D + c, u);
      Vec8<__half>::load_f32(om + ((size_t)(h * 2 + 1) * rows + prow) * D + c, w);
    }
    uint32_t mx = absmax8_bf16(raw);
#pragma unroll
    for (int o = L / 2; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    fin = fin && mx < 0x7F800000u;
    // a row of zeros, or one that is not finite, asks for nothing of the others
    const bool some = mx != 0 && mx < 0x7F800000u;
    const int e = some ? diff_exp(mx) : -kScaleMaxExp;
    const float mul = pow2f(-e);
    const __nv_bfloat162* hb = reinterpret_cast<const __nv_bfloat162*>(&raw);
    float x[8], a = 0.f, b = 0.f, ss = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(hb[k]);
      x[2 * k] = f.x * mul;
      x[2 * k + 1] = f.y * mul;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a = fmaf(x[k], u[k], a);
      b = fmaf(x[k], w[k], b);
      ss += fabsf(x[k]);
    }
#pragma unroll
    for (int o = L / 2; o; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const int nx = some ? e + (int)(__float_as_uint(ss) >> 23) - 126 : kRowNone;
    if (in && some) {
      E = max(E, e);
      X = max(X, nx);
    }
    if (threadIdx.x % L == 0) {
      delta[(size_t)h * 2 * rows + prow] = a;
      delta[(size_t)(h * 2 + 1) * rows + prow] = b;
      rowx[(size_t)h * rows + prow] = row_word(e, nx);
    }
    uint4 out;
    uint32_t* po = &out.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) po[k] = pack_f16(x[2 * k], x[2 * k + 1]);
    *reinterpret_cast<uint4*>(dos + ((size_t)h * rows + prow) * D + c) = out;
  }
  if (!fin) report_error(err, LH_ERR_DEVICE, 102);
  E = __reduce_max_sync(0xffffffffu, E);
  X = __reduce_max_sync(0xffffffffu, X);
  if (lane == 0) {
    red[0][threadIdx.x >> 5] = E;
    red[1][threadIdx.x >> 5] = X;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 8; ++k) {
      E = max(E, red[0][k]);
      X = max(X, red[1][k]);
    }
    tmax[(size_t)h * g.ntile + (t.z >> 7) + t.w] = row_word(E, X);
  }
}

template <int D>
cudaError_t bwd_t(const DiffGeom& g, const DiffTC& b, const void* dout, const void* lam, void* dq, void* dk, void* dv,
                  int* err, cudaStream_t s) {
  CUtensorMap tq, tk, tv, tdo;
  const int rows = g.ntile * 128;
  if (!make_tmap_16(&tq, b.qs, D, rows, g.H, true, 128) || !make_tmap_16(&tk, b.ks, D, rows, g.Hk, true, 128) ||
      !make_tmap_16(&tv, b.vs, D, rows, g.Hk, true, 128) || !make_tmap_16(&tdo, b.dos, D, rows, g.H, true, 128))
    return cudaErrorInvalidValue;
  const int smem = BwdLayout<D, 2>::BYTES, smem_q = BwdLayout<D, 3>::BYTES;
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = diff_kernel_ready(done[0], (const void*)k_diff_dkdv_tc<D>, smem);
  if (e != cudaSuccess) return e;
  if ((e = diff_kernel_ready(done[1], (const void*)k_diff_dq_tc<D>, smem_q)) != cudaSuccess) return e;
  const float scale = (float)(1.0 / sqrt((double)(D / 2)));
  const float c2 = (float)(1.4426950408889634 / sqrt((double)(D / 2)));
  const dim3 gp(g.ntile, g.H);
  const __nv_bfloat16 *L = (const __nv_bfloat16*)lam, *dO = (const __nv_bfloat16*)dout;
  k_diff_pack_do<D><<<gp, 256, 0, s>>>(g, dO, b.om, b.tiles, b.dos, b.delta, b.rowx, b.tmax, err);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_next(k_diff_dkdv_tc<D>, dim3(g.ntile * g.Hk), kDiffThreads, smem, s, tk, tv, tq, tdo, g, L, b.tiles, b.seq,
                  b.amax, b.rowx, b.tmax, b.lse, b.delta, (__nv_bfloat16*)dk, (__nv_bfloat16*)dv, c2, scale, err);
  if (e != cudaSuccess) return e;
  return launch_next(k_diff_dq_tc<D>, dim3(g.ntile * g.H), kDiffThreads, smem_q, s, tq, tdo, tk, tv, g, L, b.tiles, b.seq,
                     b.amax, b.rowx, b.lse, b.delta, (__nv_bfloat16*)dq, b.part, c2, scale, err);
}

}  // namespace

cudaError_t launch_diff_bwd_tc(const DiffGeom& g, const DiffTC& b, const void* dout, const void* lam, void* dq, void* dk,
                               void* dv, void* dlam, int* err, cudaStream_t s) {
  cudaError_t e = g.D == 64 ? bwd_t<64>(g, b, dout, lam, dq, dk, dv, err, s) : bwd_t<128>(g, b, dout, lam, dq, dk, dv, err, s);
  if (e != cudaSuccess) return e;
  return launch_diff_dlam(g.H, g.ntile, b.part, LH_BF16, dlam, s);
}

}  // namespace lh
