// Causal differential attention on the tensor cores: working copies and the
// forward pass (bf16 I/O; fp16 operands, fp32 accumulate).
//
//   o = A1 v - lam A2 v,  A_m = softmax(q_m k_m^T / sqrt(D/2) + causal mask)
//
// Working copies (k_diff_pack). q, k, v are copied once, from the caller's
// layout into [head][padded row][D] fp16, times a power of two per sequence and
// key/value head that brings the largest magnitude into [1/8, 256) (diff_exp):
// bf16 values enter fp16 unchanged but for that power, and P and dS may then be
// rounded to fp16's 11 bits instead of bf16's 8, which is what keeps the
// difference of two maps, and its gradients, at the accuracy of the bf16 results
// themselves. Every tile starts at a multiple of 128 rows and is filled up with
// zeros, so the kernels behind it load whole tiles by TMA whatever the strides,
// offsets and sequence ends are, and no row of another sequence is ever in one.
// A first pass copies with the power 2^0 and records the magnitudes; a second
// launch redoes the heads that need another power (others leave at once).
//
// For training both maps' outputs A_m v are kept in fp16, 11 bits where o has 8:
// the backward forms d_m = <do, A_m v> of them, and a d_m off by 2^-12 of its terms
// is below what the rounding of the gradients adds (fp32 would double what is kept).
//
// k_diff_fwd_tc. One CTA per 128-row query tile and head; both maps share the
// rows, so the second stream of tiles that keeps the tensor core busy during a
// softmax is the second map, and K and V tiles are loaded once for both.
// Three warpgroups: warp 0 TMA producer, warp 1 MMA issuer; warps 4-7 softmax of
// map 1, warps 8-11 of map 2 (one thread per row and map). TMEM: S1, O1, S2, O2, 128
// columns each. Per key tile j the issuer runs
//   PV_1(j), S_1(j+1), PV_2(j), S_2(j+1)
// (S_m: 128 x 128 x D/2, PV_m: 128 x D x 128, P_m as the TMEM operand in S_m's
// columns, handed over in two halves so that the first half's product runs under
// the second's exponentials), so one map's softmax runs under the other's
// products. The running maximum is raised only when it grows by more than 2^8; P
// is held at 2^7 times its value (both cancel in O / l), which keeps it normal in
// fp16 down to 2^-21 of the row's maximum. In the end the two warpgroups exchange
// the rows' denominators and each combines half of the columns.
// Per 128 x 128 pair of tiles: 768 * 16,384 flops against 32,768 exponentials,
// 1,536 tensor cycles against 2,048 of the special-function unit: it is the
// exponentials that bound it. Measured at 16 heads of 8,192 tokens, D = 128: 397 us,
// 1,037 TFLOP/s (440 in a long loop under the power cap), and 10 us per CTA besides the
// pairs; 3,110 cycles per pair (score wait 1,100, loads and maximum 420,
// exponentials 1,400 per map, the two maps half a turn apart). Slower: keys in
// halves of 64 with two score buffers per map (the N = 64 score products cost more
// than the waits they hide), an issuer per map, a share of the exponentials as
// polynomials on the FMA pipe; for D = 64, P behind O in tensor memory and the next
// scores formed as soon as the warps hold these (412 against 386 us: without the
// wait both maps' warps meet in the exponentials).
#include <cudaTypedefs.h>

#include "k_diff_tc.cuh"

namespace lh {
namespace {

using namespace tc;

constexpr float kPBias = 7.f;       // P is held at 2^7 times its value

// ---------------------------------------------------------------- working copies

// absmax8_bf16 of the finite ones: a value that is not finite says nothing about the
// power that the others need.
__device__ uint32_t absmax8_finite(const uint4& r) {
  uint32_t m = 0;
  for (const uint32_t w : {r.x, r.y, r.z, r.w})
    for (const uint32_t x : {(w & 0x7FFFu) << 16, w & 0x7FFF0000u}) m = max(m, x < 0x7F800000u ? x : 0);
  return m;
}

// One 128-row tile of one head of q, k or v. blockIdx.y: H query heads, then Hk
// of k, Hk of v. REDO: only the heads whose power is not 2^0.
template <bool REDO>
__global__ void __launch_bounds__(256) k_diff_pack(const DiffGeom g, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                                   const __nv_bfloat16* v, __half* qs, __half* ks, __half* vs,
                                                   const DiffTile* tiles, const int* seq, uint32_t* amax, int* err) {
  pdl_start();
  if ((int)blockIdx.x >= diff_used(tiles, g, err)) return;
  const int y = blockIdx.y;
  const int which = y < g.H ? kScaleQ : y < g.H + g.Hk ? kScaleK : kScaleV;
  const int hd = which == kScaleQ ? y : which == kScaleK ? y - g.H : y - g.H - g.Hk;
  const int hk = which == kScaleQ ? hd / g.G : hd;
  const DiffTile t = tiles[blockIdx.x];
  uint32_t* am = amax + ((size_t)which * g.B + seq[blockIdx.x]) * g.Hk + hk;
  float mul = 1.f;
  if (REDO) {
    const int e = diff_exp(*am);
    if (e == 0) return;
    mul = pow2f(-e);
  }
  const long long ld = which == kScaleQ ? g.ldq : which == kScaleK ? g.ldk : g.ldv;
  const __nv_bfloat16* src = (which == kScaleQ ? q : which == kScaleK ? k : v) + (long long)t.x * ld + (long long)hd * g.D;
  __half* dst = (which == kScaleQ ? qs : which == kScaleK ? ks : vs) +
                ((size_t)hd * g.ntile * kDiffTileTC + t.z + t.w * kDiffTileTC) * g.D;
  const int nv = g.D / 8, r0 = t.w * kDiffTileTC;
  uint32_t mx = 0;
  bool fin = true;
#pragma unroll 4
  for (int i = threadIdx.x; i < kDiffTileTC * nv; i += 256) {
    const int r = i / nv, c = (i - r * nv) * 8;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (r0 + r < t.y) raw = __ldg(reinterpret_cast<const uint4*>(src + (long long)(r0 + r) * ld + c));
    if (!REDO) mx = max(mx, absmax8_bf16(raw));
    uint4 out;
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(h[e]);
      o[e] = pack_f16(f.x * mul, f.y * mul);
    }
    *reinterpret_cast<uint4*>(dst + (size_t)r * g.D + c) = out;
  }
  if (!REDO) {
    if (mx >= 0x7F800000u) {           // rare: the thread's values once more
      fin = false;
      mx = 0;
      for (int i = threadIdx.x; i < kDiffTileTC * nv; i += 256) {
        const int r = i / nv, c = (i - r * nv) * 8;
        if (r0 + r < t.y) mx = max(mx, absmax8_finite(__ldg(reinterpret_cast<const uint4*>(src + (long long)(r0 + r) * ld + c))));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((threadIdx.x & 31) == 0 && mx > *am) atomicMax(am, mx);
    if (!fin) report_error(err, LH_ERR_DEVICE, 102);
  }
}

// ---------------------------------------------------------------- forward

template <int D>
struct FwdLayout {
  static constexpr int SUB = D / 64;
  static constexpr int OPB = SUB * kDSub;    // one 128-row operand tile
  static constexpr int NST = 3;              // stages of K and of V
  static constexpr int Q = 0;
  static constexpr int K = Q + OPB;
  static constexpr int V = K + NST * OPB;
  static constexpr int TILES = V + NST * OPB;
  static constexpr int HEAD = 256 + 2 * 128 * 4;   // barriers, then both maps' 1 / l
  static constexpr int BYTES = HEAD + 1024 + TILES;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

struct FwdBars {
  uint64_t q_full, k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], drain;
  uint32_t tmem_base;
  Abort abort;
};
static_assert(sizeof(FwdBars) <= 256, "barrier block");

template <int D>
__global__ void __launch_bounds__(kDiffThreads, 1)
k_diff_fwd_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              const __grid_constant__ CUtensorMap tv, const DiffGeom g, const __nv_bfloat16* __restrict__ lam,
              const DiffTile* __restrict__ tiles, const int* __restrict__ seq, const uint32_t* __restrict__ amax,
              __nv_bfloat16* __restrict__ o, __half* __restrict__ om, float* __restrict__ lse, float c2, int* err) {
  using Lay = FwdLayout<D>;
  constexpr int SUB = Lay::SUB, NST = Lay::NST, KS = D / 32;     // 16-wide steps of one map's score product
  constexpr uint32_t IDS = idesc_f16(128, 128, false);           // S = Q K^T, both K-major
  constexpr uint32_t IDO = idesc_f16(128, D, true);              // O = P V, V MN-major
  extern __shared__ __align__(16) uint8_t smem_raw[];
  FwdBars* bars = reinterpret_cast<FwdBars*>(smem_raw);
  float* linv = reinterpret_cast<float*>(smem_raw + 256);        // [2][128]
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + Lay::HEAD + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(sm);
  int rank, h;
  diff_place(g.oq, blockIdx.x, rank, h);
  const int hk = h / g.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_map(&tq);
    prefetch_map(&tk);
    prefetch_map(&tv);
  }
  pdl_start();
  TileLoad tl;
  tl.ask(tiles, seq, g, rank);
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_half[s], 4);
      mbar_init(&bars->p_full[s], 4);
      mbar_init(&bars->o_done[s], 1);
    }
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
  const uint32_t tbase = bars->tmem_base;
  volatile Abort* ab = &bars->abort;
  if (!tl.live(g, rank, err)) {                                  // the whole CTA
    if (warp == 1) tmem_dealloc(tbase, 512);
    return;
  }
  const DiffTile t = tl.t;
  const int nkv = t.w + 1;

  if (warp < 4) regs_give();
  if (warp == 0) {
    if (lane == 0) {
      int ik = 0, iv = 0;            // K / V tiles issued
      mbar_expect_tx(&bars->q_full, Lay::OPB);
      for (int c = 0; c < SUB; ++c)
        tma_load_3d(sm + Lay::Q + c * kDSub, &tq, &bars->q_full, 64 * c, t.z + t.w * 128, h);
      for (int j = 0; j < nkv; ++j) {
        const int st = j % NST;
        if (j >= NST && !mbar_wait(&bars->k_empty[st], ((j / NST) - 1) & 1, ab, err, 31)) break;
        mbar_expect_tx(&bars->k_full[st], Lay::OPB);
        for (int c = 0; c < SUB; ++c)
          tma_load_3d(sm + Lay::K + st * Lay::OPB + c * kDSub, &tk, &bars->k_full[st], 64 * c, t.z + j * 128, hk);
        ik = j + 1;
        if (j >= NST && !mbar_wait(&bars->v_empty[st], ((j / NST) - 1) & 1, ab, err, 31)) break;
        mbar_expect_tx(&bars->v_full[st], Lay::OPB);
        for (int c = 0; c < SUB; ++c)
          tma_load_3d(sm + Lay::V + st * Lay::OPB + c * kDSub, &tv, &bars->v_full[st], 64 * c, t.z + j * 128, hk);
        iv = j + 1;
      }
      if (ab->flag) {
        // wind-down: let the copies still in flight land before the CTA exits
        Abort none{0};
        mbar_wait(&bars->q_full, 0, &none, nullptr, 0);
        for (int j = ik - NST < 0 ? 0 : ik - NST; j < ik; ++j)
          mbar_wait(&bars->k_full[j % NST], (j / NST) & 1, &none, nullptr, 0);
        for (int j = iv - NST < 0 ? 0 : iv - NST; j < iv; ++j)
          mbar_wait(&bars->v_full[j % NST], (j / NST) & 1, &none, nullptr, 0);
      }
    }
  } else if (warp == 1) {
    const bool leader = elect_one();
    constexpr uint32_t OPB16 = Lay::OPB >> 4;
    const uint64_t dQ = sdesc_sw128(sbase + Lay::Q, 16, 1024), dK = sdesc_sw128(sbase + Lay::K, 16, 1024);
    const uint64_t dV = sdesc_sw128(sbase + Lay::V, kDSub, 1024);
    auto issue_s = [&](int m, int j) {       // S_m = Q_m K_m^T: steps m KS .. of the row's 16-wide slices
      const uint64_t b0 = dK + (uint64_t)((j % NST) * OPB16);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
          umma_f16(tbase + 256 * m, dQ + kslice(m * KS + kk), b0 + kslice(m * KS + kk), IDS, kk > 0 ? 1u : 0u);
        umma_commit(&bars->s_full[m]);
      }
    };
    auto issue_pv = [&](int m, int j, int half) {      // O_m += P_m V, 64 keys of the tile
      const uint64_t b0 = dV + (uint64_t)((j % NST) * OPB16);
      const uint32_t tS = tbase + 256 * m, tO = tS + 128;
      if (leader) {
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kk = 4 * half + k4;
          umma_f16_ts(tO, tS + 32 * (kk >> 1) + 8 * (kk & 1), b0 + kk * 128, IDO, (j > 0 || kk > 0) ? 1u : 0u);
        }
        if (half) umma_commit(&bars->o_done[m]);
      }
    };
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, err, site));
    };
    bool ok = wait(&bars->q_full, 0, 32) && wait(&bars->k_full[0], 0, 33);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      issue_s(1, 0);
      if (leader) umma_commit(&bars->k_empty[0]);
    }
    for (int j = 0; ok && j < nkv; ++j) {
      const bool more = j + 1 < nkv;
      if (!wait(&bars->v_full[j % NST], (j / NST) & 1, 34)) { ok = false; break; }
      if (!wait(&bars->p_half[0], j & 1, 35)) { ok = false; break; }
      tc_fence_after();
      issue_pv(0, j, 0);
      if (!wait(&bars->p_full[0], j & 1, 35)) { ok = false; break; }
      tc_fence_after();
      issue_pv(0, j, 1);
      if (more) {
        if (!wait(&bars->k_full[(j + 1) % NST], ((j + 1) / NST) & 1, 33)) { ok = false; break; }
        tc_fence_after();
        issue_s(0, j + 1);
      }
      if (!wait(&bars->p_half[1], j & 1, 35)) { ok = false; break; }
      tc_fence_after();
      issue_pv(1, j, 0);
      if (!wait(&bars->p_full[1], j & 1, 35)) { ok = false; break; }
      tc_fence_after();
      issue_pv(1, j, 1);
      if (leader) umma_commit(&bars->v_empty[j % NST]);
      if (more) {
        issue_s(1, j + 1);
        if (leader) umma_commit(&bars->k_empty[(j + 1) % NST]);
      }
    }
    // wait until every MMA issued here has finished before TMEM is released
    if (leader) umma_commit(&bars->drain);
    __syncwarp();
    Abort none{0};
    mbar_wait(&bars->drain, 0, &none, nullptr, 0);
  } else if (warp >= 4) {
    regs_take();
    // softmax of map m: one thread per query row / TMEM lane
    const int m = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t la = (uint32_t)(quarter * 32) << 16;
    const uint32_t cS = tbase + la + 256 * m, cO = cS + 128;
    const int row = t.w * 128 + r;                       // within the sequence
    const uint32_t* am = amax + (size_t)tl.b * g.Hk + hk;
    const size_t plane = (size_t)g.B * g.Hk;
    const int ev = diff_exp(am[kScaleV * plane]);
    c2 *= pow2f(diff_exp(am[kScaleQ * plane]) + diff_exp(am[kScaleK * plane]));
    float m_run = 0.f, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[m], j & 1, ab, err, 36))) { ok = false; break; }
      tc_fence_after();
      uint32_t s[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(cS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
      tmem_wait_ld_regs(*reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&s[32]));
      reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&s[64]));
      reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&s[96]));
      // the diagonal tile: columns past the row's own position. Key 0 is in
      // every row's first tile, so a running maximum is finite from there on.
      if (j == t.w) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > r) s[c] = __float_as_uint(-INFINITY);
      }
      // eight strands, so that the chain of dependent maxima is short
      float mq[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        mq[q] = __uint_as_float(s[16 * q]);
#pragma unroll
        for (int c = 1; c < 15; c += 2)
          mq[q] = fmax3(mq[q], __uint_as_float(s[16 * q + c]), __uint_as_float(s[16 * q + c + 1]));
        mq[q] = fmaxf(mq[q], __uint_as_float(s[16 * q + 15]));
      }
      const float mx = fmaxf(fmax3(fmax3(mq[0], mq[1], mq[2]), mq[3], mq[4]), fmax3(mq[5], mq[6], mq[7])) * c2;
      float m_new = m_run, alpha = 1.f;
      if (j == 0) {
        m_new = mx;
      } else if (mx > m_run + 8.f) {
        m_new = mx;
        alpha = ex2(m_run - m_new);
      }
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
        // O_m is current: PV_m(j-1) finished before S_m(j) (same MMA stream)
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t x[16];
          tmem_ld16(cO + 16 * c, x);
          tmem_wait_ld_regs16(x);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
          tmem_st16(cO + 16 * c, x);
        }
      }
      const float2 cc = make_float2(c2, c2), nm = make_float2(kPBias - m_new, kPBias - m_new);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __ffma2_rn(
              make_float2(__uint_as_float(s[32 * c + 2 * e]), __uint_as_float(s[32 * c + 2 * e + 1])), cc, nm);
          const float2 pp = make_float2(ex2(x.x), ex2(x.y));
          acc[e & 1] = __fadd2_rn(acc[e & 1], pp);
          const __half2 p2 = __float22half2_rn(pp);
          pk[e] = *reinterpret_cast<const uint32_t*>(&p2);
        }
        tmem_st16(cS + 32 * c, pk);
        if (c == 1) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_warp(&bars->p_half[m]);
        }
      }
      const float2 a01 = __fadd2_rn(acc[0], acc[1]);
      l_run = l_run * alpha + (a01.x + a01.y);
      m_run = m_new;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive_warp(&bars->p_full[m]);
    }
    linv[m * 128 + r] = 1.f / l_run;
    named_bar_sync(1, 256);              // every softmax thread comes here, after a wind-down too
    // PV_m(nkv-2) finished before S_m(nkv-1): phase nkv-1 is the one left
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->o_done[0], (nkv - 1) & 1, ab, err, 38));
    ok = ok && __all_sync(0xffffffffu, mbar_wait(&bars->o_done[1], (nkv - 1) & 1, ab, err, 38));
    if (ok) {
      tc_fence_after();
      const float i0 = linv[r], i1 = linv[128 + r];
      const float lm = __bfloat162float(lam[h]), pv = pow2f(ev);
      const bool in = row < t.y;
      const size_t prow = (size_t)h * 2 * g.ntile * 128 + t.z + row;      // [H][2][padded rows]
      // this warpgroup's half of the columns, by way of the tiles' shared memory
      // (every product and so every copy into it is done)
      constexpr int CH = D / 16, BUF = 32 * CH * 16;
      uint8_t* buf = sm + (warp - 4) * 3 * BUF;
#pragma unroll 1
      for (int c = m * (D / 64); c < (m + 1) * (D / 64); ++c) {
        uint32_t a[32], b[32];
        tmem_ld32(tbase + la + 128 + 32 * c, a);
        tmem_ld32(tbase + la + 384 + 32 * c, b);
        tmem_wait_ld_regs(a);
        reg_fence32(b);
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint4 both, u, w;
          uint32_t *pb = &both.x, *pu = &u.x, *pw = &w.x;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float x0 = __uint_as_float(a[e + 2 * x]) * i0, x1 = __uint_as_float(a[e + 2 * x + 1]) * i0;
            const float y0 = __uint_as_float(b[e + 2 * x]) * i1, y1 = __uint_as_float(b[e + 2 * x + 1]) * i1;
            pb[x] = pack_bf16(fmaf(-lm, y0, x0) * pv, fmaf(-lm, y1, x1) * pv);
            pu[x] = pack_f16(x0, x1);
            pw[x] = pack_f16(y0, y1);
          }
          const int piece = 4 * (c - m * (D / 64)) + e / 8;
          put_piece<CH>(buf, lane, piece, both);
          if (om) {
            put_piece<CH>(buf + BUF, lane, piece, u);
            put_piece<CH>(buf + 2 * BUF, lane, piece, w);
          }
        }
      }
      __syncwarp();
      const int first = t.w * 128 + quarter * 32, live = t.y - first;
      put_rows<CH>(buf, lane, o + (long long)(t.x + first) * g.ldo + (long long)h * D + m * (D / 2), g.ldo, live);
      if (om) {
        __half* d0 = om + ((size_t)h * 2 * g.ntile * 128 + t.z + first) * D + m * (D / 2);
        put_rows<CH>(buf + BUF, lane, d0, D, live);
        put_rows<CH>(buf + 2 * BUF, lane, d0 + (size_t)g.ntile * 128 * D, D, live);
      }
      if (lse && in) lse[prow + (size_t)m * g.ntile * 128] = m_run + log2f(l_run) - kPBias;      // base 2
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

template <int D>
cudaError_t fwd_t(const DiffGeom& g, const DiffTC& b, const void* lam, void* o, int train, int* err, cudaStream_t s) {
  CUtensorMap tq, tk, tv;
  const int rows = g.ntile * 128;
  if (!make_tmap_16(&tq, b.qs, D, rows, g.H, true, 128) || !make_tmap_16(&tk, b.ks, D, rows, g.Hk, true, 128) ||
      !make_tmap_16(&tv, b.vs, D, rows, g.Hk, true, 128))
    return cudaErrorInvalidValue;
  const int smem = FwdLayout<D>::BYTES;
  auto kern = k_diff_fwd_tc<D>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = diff_kernel_ready(done, (const void*)kern, smem);
  if (e != cudaSuccess) return e;
  const float c2 = (float)(1.4426950408889634 / sqrt((double)(D / 2)));
  return launch_next(kern, dim3(g.ntile * g.H), kDiffThreads, smem, s, tq, tk, tv, g, (const __nv_bfloat16*)lam, b.tiles,
                     b.seq, b.amax, (__nv_bfloat16*)o, train ? b.om : nullptr, train ? b.lse : nullptr, c2, err);
}

}  // namespace

cudaError_t launch_diff_fwd_tc(const DiffGeom& g, const DiffTC& b, const void* q, const void* k, const void* v,
                               const void* lam, void* o, int train, int* err, cudaStream_t s) {
  cudaError_t e = launch_diff_tiles(g, kDiffTileTC, b.tiles, b.seq, b.amax, err, s);
  if (e != cudaSuccess) return e;
  const dim3 grid(g.ntile, g.H + 2 * g.Hk);
  for (auto kern : {k_diff_pack<false>, k_diff_pack<true>}) {
    e = launch_next(kern, grid, 256, 0, s, g, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, b.qs,
                    b.ks, b.vs, b.tiles, b.seq, b.amax, err);
    if (e != cudaSuccess) return e;
  }
  return g.D == 64 ? fwd_t<64>(g, b, lam, o, train, err, s) : fwd_t<128>(g, b, lam, o, train, err, s);
}

}  // namespace lh
