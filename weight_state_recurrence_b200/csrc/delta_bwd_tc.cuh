// Backward of the gated delta rule on the 5th-generation tensor cores (bf16,
// d_k and d_v in {64, 128}), over the chunks and records of delta_tc.cuh.
//
// With S0 the state before a chunk, D the gradient that reaches the state
// after it, X = V - e^gamma K S0 and r, u = beta r as in the forward:
//   dU = e^(gamma_C - gamma) K D + P^T dO,     du = dU + G^T (beta dU)
//   dv = beta du,                              dbeta = rowsum(du o r)
//   D <- e^gamma_C D + Q^T (e^gamma dO) - K^T (e^gamma beta du)
//   M = Gam o (dO u^T) (s <= t),   Y = Gam o ((beta du) u^T) (s < t)
//   dq = e^gamma dO S0^T + M K
//   dk = e^(gamma_C - gamma) u D^T + M^T Q - (Y + Y^T) K - e^gamma (beta du) S0^T
// and dg_i sums what passes token i, as in delta_simt.cuh.
//
// The recurrence of S forwards and that of D backwards do not need each other:
// both run in one launch, a CTA per head and direction (sweep), and keep the
// states of every chunk and r, du of every token, as bf16 pairs.  Then every
// chunk is done at once (grad).
#pragma once
#include "delta_tc.cuh"

namespace linattn {
namespace delta {

// What the sweeps keep, each as a hi and a lo array of bf16: states
// [B H chunks, d_v, d_k] (transposed, as the sweeps hold them), rows [B H, N, d_v].
// The recurrences themselves hold S and D in fp32; what is kept are the pairs that
// the products of the gradients take in any case.
struct Kept {
  __nv_bfloat16 *s_hi, *s_lo;   // S before the chunk
  __nv_bfloat16 *d_hi, *d_lo;   // D after the chunk
};

// ------------------------------------------------------------------ sweep
namespace sweep {

// The chain of delta_tc.cuh without outputs, in either direction: everything
// transposed, a TMEM lane to a column of the state.
//   forward:  pre = V^T,      x = -e^gamma (S^T k^T),            r = pre + x + ..
//   reverse:  pre = dO^T P,   x = e^(gamma_C - gamma) (D^T k^T),  du likewise
//   pairs of beta (pre + x), by G (forward) or its transpose, added to pre
//   state += f (pre + x) k,   f = beta e^(gamma_C - gamma), or -beta e^gamma,
//   and in the reverse (e^gamma dO)^T q, whose left operand the output warps
//   make out of dO^T while the chain is elsewhere.
// The state's pairs are kept once a chunk, 64 KB of them: through the stage of
// the chunk that has just been read, whose k, q, v and G they may overwrite,
// and on by bulk stores (warp 2).  64 heads x 2048 tokens: 160 us, 164 with
// stores by the lanes, each to a row of its own, 130 without keeping them; all
// that the sweeps read and write there takes 117 us at the copy rate.  With d_k = 128
// the 80 registers of 24 warps spill 192 bytes a thread.
constexpr int NT = 768;
constexpr uint32_t kOffKQ = 0;
constexpr uint32_t kOffV = 2 * kPanelKQ;
constexpr uint32_t kOffRec = kOffV + 2 * kTileHalf;
constexpr uint32_t kStage = kOffRec + kRecord;
constexpr int kStages = 2;
constexpr uint32_t kOffOut = kStages * kStage;          // 3 tiles [64, d_v]: hi, lo, dv
constexpr uint32_t kOffEye = kOffOut + 6 * kTileHalf;
constexpr uint32_t kOffBar = kOffEye + kTileHalf;
constexpr uint32_t kSmemBytes = kOffBar + 256;
static_assert(kSmemBytes <= 232448, "exceeds the per-CTA shared memory of sm_100");
static_assert(kStage % 1024 == 0, "tiles start on 1024 bytes");
static_assert(kOffRec + kRecP == 4 * kPanelKQ, "a state's pairs take the place of k, q, v and G");

enum Bar {
  kFull0 = 0, kFull1, kFree0, kFree1,
  kKS, kGX, kS, kAux,                                    // products
  kXReady, kUdReady, kSReady, kScaled, kRReady,          // chain warps
  kAuxReady, kRFree, kOutFree0, kOutFree1,               // output warps
  kKept, kStored0, kStored1,   // the next state is in the stage; and on its way
  kFinal, kNumBars
};
constexpr uint32_t kOffTmem = 224;
static_assert(kNumBars * 8 <= 224, "barrier area overflow");

constexpr uint32_t kTmS = 0, kTmSh = 128, kTmSl = 192;
constexpr uint32_t kTmX = 256;    // state^T k^T; then the pairs of beta (pre + x)
constexpr uint32_t kTmG = 320;    // pre, and its product by G; then the state's pairs
constexpr uint32_t kTmR = 384;    // r or du, fp32, for the output warps
constexpr uint32_t kTmA = 448;    // dO^T; then the pairs of e^gamma dO^T
constexpr uint32_t kTmCols = 512;

struct Args {
  const uint8_t *rec;
  const float *init;                  // S_init or dS_final
  float *last;                        // dS_init (reverse), or NULL
  __nv_bfloat16 *keep_hi, *keep_lo;   // the state at every chunk
  int nch, dv;
};

template <int DKP, bool REV>
__device__ __forceinline__ void run(uint8_t *sm, const CUtensorMap *tm_q, const CUtensorMap *tm_k,
                                    const CUtensorMap *tm_v, const CUtensorMap *tm_hi,
                                    const CUtensorMap *tm_lo, const CUtensorMap *tm_dv,
                                    const CUtensorMap *tm_kh, const CUtensorMap *tm_kl, const Args &a,
                                    long head) {
  constexpr int DK = 64 * DKP;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int nch = a.nch, dv = a.dv;
  auto bar = [&](int i) { return sb + kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + kOffTmem);
  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bar(i), (i >= kXReady && i <= kRReady) || i == kKept ? 16
                        : i >= kAuxReady && i <= kOutFree1           ? 4
                                                                     : 1);
    fence_mbar_init();
  }
  for (int i = tid; i < C * C / 2; i += NT) {
    const uint32_t r = i / (C / 2), e = 2 * (i % (C / 2));
    *reinterpret_cast<uint32_t *>(sm + kOffEye + sw128_offset(r, e * 2)) =
        r == e ? 0x00003f80u : r == e + 1 ? 0x3f800000u : 0u;
  }
  if (dv == 64)
    for (int s = 0; s < kStages; ++s)
      for (uint32_t i = tid * 16; i < kTileHalf; i += NT * 16)
        *reinterpret_cast<uint4 *>(sm + s * kStage + kOffV + kTileHalf + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();   // prep
  // a wait that runs out: as in the chain of delta_tc.cuh
  auto wait = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity & 1); };
  bool ok = true;
  auto pass = [&](int i, uint32_t parity) {
    if (ok) ok = wait(i, parity);
    tc_fence_after();
  };
  auto chunk = [&](int c) { return REV ? nch - 1 - c : c; };   // of step c

  if (warp == 0) {
    if (lane == 0) {
      const int vp = dv / 64;
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1, z = static_cast<int>(head), y = chunk(c) * C;
        const uint32_t st = sb + s * kStage, full = bar(kFull0 + s);
        const uint8_t *r = a.rec + (head * nch + chunk(c)) * kRecord;
        if (c >= kStages && (!wait(kFree0 + s, (c >> 1) + 1) || !wait(kOutFree0 + s, (c >> 1) + 1) ||
                             !wait(kStored0 + s, (c >> 1) + 1)))
          break;
        mbar_arrive_expect_tx(full, ((REV ? 2 : 1) * DKP + vp + (REV ? 4 : 2)) * kTileHalf + kScalBytes);
        for (int p = 0; p < DKP; ++p) {
          const uint32_t t = st + kOffKQ + p * kPanelKQ;
          tma_load_3d(t, tm_k, full, 64 * p, y, z);
          if (REV) tma_load_3d(t + kTileHalf, tm_q, full, 64 * p, y, z);
        }
        for (int p = 0; p < vp; ++p)
          tma_load_3d(st + kOffV + p * kTileHalf, tm_v, full, 64 * p, y, z);
        bulk_load(st + kOffRec + kRecScal, r + kRecScal, kScalBytes, full);
        bulk_load(st + kOffRec + kRecG, r + kRecG, (REV ? 4 : 2) * kTileHalf, full);
        issued = c + 1;
      }
      // the copies this thread started have to land before the CTA exits
      for (int c = issued - kStages < 0 ? 0 : issued - kStages; c < issued; ++c)
        mbar_wait(bar(kFull0 + (c & 1)), (c >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idC = idesc_bf16(128, C, 0, 0);     // k: K-major, N = C
      constexpr uint32_t idK = idesc_bf16(128, DK, 0, 1);    // k, q as [C, d_k]: MN-major
      constexpr uint32_t idV = idesc_bf16(128, C, 1, 0);     // v, dO as [C, d_v]: MN-major
      constexpr uint32_t idVP = idesc_bf16(128, C, 1, 1);    // ... by P, contracted over its rows
      const uint64_t dK = sdesc_sw128(sb + kOffKQ, 16, 1024);
      const uint64_t dKmn = sdesc_sw128(sb + kOffKQ, kPanelKQ, 1024);
      const uint64_t dV = sdesc_sw128(sb + kOffV, kTileHalf, 1024);
      const uint64_t dG = sdesc_sw128(sb + kOffRec + kRecG, 16, 1024);
      const uint64_t dP = sdesc_sw128(sb + kOffRec + kRecP, 16, 1024);
      const uint64_t dEye = sdesc_sw128(sb + kOffEye, 16, 1024);
      auto state_add = [&](uint32_t pairs, uint64_t b) {
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            umma_bf16_ts(tmem + kTmS, tmem + pairs + pair_col(ks, term), b + ((ks * 2048) >> 4), idK, 1u);
      };
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        const uint64_t so = static_cast<uint64_t>(s) * (kStage >> 4);
        if (!wait(kFull0 + s, c >> 1)) break;
        tc_fence_after();
        if constexpr (REV) {
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int ks = 0; ks < C / 16; ++ks)
              umma_bf16(tmem + kTmG, dV + so + ((ks * 2048) >> 4),
                        dP + so + ((term * kTileHalf + ks * 2048) >> 4), idVP, term + ks > 0);
        }
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          umma_bf16(tmem + (REV ? kTmA : kTmG), dV + so + ((ks * 2048) >> 4), dEye + ((ks * 32) >> 4),
                    idV, ks > 0);
        if constexpr (REV) umma_commit(bar(kAux));
        if (!wait(kSReady, c)) break;
        tc_fence_after();
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < 4 * DKP; ++ks)
            umma_bf16_ts(tmem + kTmX, tmem + (term ? kTmSl : kTmSh) + 8 * ks,
                         dK + so + (((ks >> 2) * kPanelKQ + (ks & 3) * 32) >> 4), idC, term + ks > 0);
        umma_commit(bar(kKS));
        if (!wait(kXReady, c)) break;
        tc_fence_after();
        pairs_hi<REV>(tmem, kTmG, kTmX, dG + so, true);
        pairs_lo<REV>(tmem, kTmG, kTmX, dG + so);
        umma_commit(bar(kGX));
        if constexpr (REV) {
          if (!wait(kAuxReady, c) || !wait(kScaled, c)) break;
          tc_fence_after();
          state_add(kTmA, dKmn + so + (kTileHalf >> 4));
        }
        if (!wait(kUdReady, c)) break;
        tc_fence_after();
        state_add(kTmG, dKmn + so);
        umma_commit(bar(kS));
        umma_commit(bar(kFree0 + s));
      }
      umma_commit(bar(kFinal));
      mbar_wait(bar(kFinal), 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {
      for (int c = 0; c + 1 < nch; ++c) {
        if (!wait(kKept, c)) break;
        const int plane = static_cast<int>(head * nch + chunk(c + 1));
        for (int p = 0; p < DKP; ++p)
          for (int v = 0; v < dv / 64; ++v) {
            const uint32_t t = sb + (c & 1) * kStage + p * kPanelKQ + v * kTileHalf;
            tma_store_3d(tm_kh, t, 64 * p, 64 * v, plane);
            tma_store_3d(tm_kl, t + 2 * kPanelKQ, 64 * p, 64 * v, plane);
          }
        tma_store_commit();
        tma_store_wait_read();
        mbar_arrive(bar(kStored0 + (c & 1)));
      }
      tma_store_wait_all();
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 20) {
    const int wq = warp & 3, h = (warp - 4) >> 2;
    const int col = wq * 32 + lane;                     // column of the state
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    constexpr int SC = DK / 4;                          // d_k columns per warp
    const int k0 = h * SC, t0 = 16 * h;
    auto arrive = [&](int i) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    auto scal = [&](int c) {
      return reinterpret_cast<const float *>(sm + (c & 1) * kStage + kOffRec + kRecScal);
    };
    // the pairs of this warp's columns of the state
    auto put_pairs = [&](const uint32_t (&v)[SC]) {
#pragma unroll
      for (int j = 0; j < SC; j += 16) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2(as_f2(v[j + 2 * i], v[j + 2 * i + 1]), hi[i], lo[i]);
        tmem_st<8>(tmem + lf + kTmSh + (k0 + j) / 2, hi);
        tmem_st<8>(tmem + lf + kTmSl + (k0 + j) / 2, lo);
      }
    };
    // ... and out of TMEM again: the first state to memory, the others into
    // the stage of chunk c while the product with k runs
    auto keep_first = [&]() {
      const long at = ((head * nch + chunk(0)) * dv + col) * DK + k0;
#pragma unroll
      for (int j = 0; j < SC; j += 16) {
        uint32_t hi[8], lo[8];
        tmem_ld_32x32b_x8(tmem + lf + kTmSh + (k0 + j) / 2, hi);
        tmem_ld_32x32b_x8(tmem + lf + kTmSl + (k0 + j) / 2, lo);
        tmem_wait_ld();
        if (live) {
          st_global_na_v8(a.keep_hi + at + j, hi);
          st_global_na_v8(a.keep_lo + at + j, lo);
        }
      }
    };
    auto keep_pairs = [&](int c) {
      uint8_t *t = sm + (c & 1) * kStage;
#pragma unroll
      for (int j = 0; j < SC; j += 16) {
        uint32_t hi[8], lo[8];
        tmem_ld_32x32b_x8(tmem + lf + kTmSh + (k0 + j) / 2, hi);
        tmem_ld_32x32b_x8(tmem + lf + kTmSl + (k0 + j) / 2, lo);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t o = ((k0 + j) >> 6) * kPanelKQ + sw128_offset(col, ((k0 + j) & 63) * 2 + 16 * i);
          *reinterpret_cast<uint4 *>(t + o) =
              make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
          *reinterpret_cast<uint4 *>(t + 2 * kPanelKQ + o) =
              make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kKept));
    };
    auto put_scaled = [&](uint32_t (&v)[SC], const float *scal) {
      scale_state(v, scal);
      tmem_st<SC>(tmem + lf + kTmS + k0, v);
    };
    pass(kFull0, 0);
    {
      uint32_t v[SC];
#pragma unroll
      for (int i = 0; i < SC; ++i)
        v[i] = a.init && live ? __float_as_uint(a.init[(head * DK + k0 + i) * dv + col]) : 0u;
      put_pairs(v);
      arrive(kSReady);
      put_scaled(v, scal(0));
      arrive(kScaled);
      keep_first();
    }
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const float *eg = scal(c) + t0, *el = eg + C, *be = el + C;
      float2 x[8];
      pass(kKS, c);
      {
        uint32_t d[16], v[16], p[16];
        tmem_ld<16>(tmem + lf + kTmX + t0, d);
        tmem_ld<16>(tmem + lf + kTmG + t0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e = *reinterpret_cast<const float4 *>((REV ? el : eg) + i);
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          constexpr float sg = REV ? 1.f : -1.f;
          x[i / 2] = fmul2(make_float2(sg * e.x, sg * e.y), as_f2(d[i], d[i + 1]));
          x[i / 2 + 1] = fmul2(make_float2(sg * e.z, sg * e.w), as_f2(d[i + 2], d[i + 3]));
          split2(fmul2(make_float2(b.x, b.y), fadd2(x[i / 2], as_f2(v[i], v[i + 1]))), p[i / 2],
                 p[8 + i / 2]);
          split2(fmul2(make_float2(b.z, b.w), fadd2(x[i / 2 + 1], as_f2(v[i + 2], v[i + 3]))),
                 p[i / 2 + 1], p[8 + i / 2 + 1]);
        }
        tmem_st<16>(tmem + lf + kTmX + t0, p);
      }
      arrive(kXReady);
      pass(kGX, c);
      {
        uint32_t d[16], p[16];
        tmem_ld<16>(tmem + lf + kTmG + t0, d);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          const float4 e = *reinterpret_cast<const float4 *>((REV ? eg : el) + i);
          constexpr float sg = REV ? -1.f : 1.f;
          x[i / 2] = fadd2(x[i / 2], as_f2(d[i], d[i + 1]));
          x[i / 2 + 1] = fadd2(x[i / 2 + 1], as_f2(d[i + 2], d[i + 3]));
          split2(fmul2(make_float2(sg * b.x * e.x, sg * b.y * e.y), x[i / 2]), p[i / 2], p[8 + i / 2]);
          split2(fmul2(make_float2(sg * b.z * e.z, sg * b.w * e.w), x[i / 2 + 1]), p[i / 2 + 1],
                 p[8 + i / 2 + 1]);
        }
        tmem_st<16>(tmem + lf + kTmG + t0, p);
      }
      arrive(kUdReady);
      if (c > 0) pass(kRFree, c - 1);
      {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[2 * i] = __float_as_uint(x[i].x);
          p[2 * i + 1] = __float_as_uint(x[i].y);
        }
        tmem_st<16>(tmem + lf + kTmR + t0, p);
      }
      arrive(kRReady);
      pass(kS, c);
      uint32_t v[SC];
      tmem_ld<SC>(tmem + lf + kTmS + k0, v);
      tmem_wait_ld();
      if (c + 1 < nch) {
        put_pairs(v);
        arrive(kSReady);
        pass(kFull0 + (s ^ 1), (c + 1) >> 1);
        put_scaled(v, scal(c + 1));
        arrive(kScaled);
        keep_pairs(c);
      } else if (a.last && live) {
#pragma unroll
        for (int i = 0; i < SC; ++i)
          a.last[(head * DK + k0 + i) * dv + col] = __uint_as_float(v[i]);
      }
    }
    tc_fence_before();
  } else if (warp >= 20) {
    const int wq = warp & 3;
    const int col = wq * 32 + lane;
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    uint8_t *ot = sm + kOffOut + (col >> 6) * kTileHalf + (col & 7) * 2;
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (((col & 63) >> 3) ^ i) << 4;
    auto put = [&](int tile, int t, uint32_t w) {   // tokens t, t + 1 of this column
      uint8_t *p = ot + tile * 2 * kTileHalf + t * 128;
      *reinterpret_cast<uint16_t *>(p + o[t & 7]) = static_cast<uint16_t>(w);
      *reinterpret_cast<uint16_t *>(p + 128 + o[(t + 1) & 7]) = static_cast<uint16_t>(w >> 16);
    };
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const float *eg = reinterpret_cast<const float *>(sm + s * kStage + kOffRec + kRecScal);
      const float *be = eg + 2 * C;
      pass(kFull0 + s, c >> 1);
      if constexpr (REV) {
        pass(kAux, c);
#pragma unroll 1
        for (int b = 0; b < C; b += 16) {
          uint32_t d[16], p[16];
          tmem_ld<16>(tmem + lf + kTmA + b, d);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(eg + b + i);
            split2(fmul2(make_float2(e.x, e.y), as_f2(d[i], d[i + 1])), p[i / 2], p[8 + i / 2]);
            split2(fmul2(make_float2(e.z, e.w), as_f2(d[i + 2], d[i + 3])), p[i / 2 + 1],
                   p[8 + i / 2 + 1]);
          }
          tmem_st<16>(tmem + lf + kTmA + b, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kAuxReady));
      }
      pass(kRReady, c);
      if (warp == 20 && lane == 0) tma_store_wait_read();
      named_bar_sync(1, 128);
#pragma unroll 1
      for (int b = 0; b < C; b += 32) {
        uint32_t d[32];
        tmem_ld<32>(tmem + lf + kTmR + b, d);
        tmem_wait_ld();
        if (live)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 f = as_f2(d[i], d[i + 1]);
            uint32_t hi, lo;
            split2(f, hi, lo);
            put(0, b + i, hi);
            put(1, b + i, lo);
            if (REV) put(2, b + i, pack2(be[b + i] * f.x, be[b + i + 1] * f.y));
          }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(kRFree));
        mbar_arrive(bar(kOutFree0 + s));
      }
      named_bar_sync(1, 128);
      if (ok && warp == 20 && lane == 0) {
        for (int p = 0; p < dv / 64; ++p) {
          const uint32_t t = sb + kOffOut + p * kTileHalf;
          const int y = chunk(c) * C, z = static_cast<int>(head);
          tma_store_3d(tm_hi, t, 64 * p, y, z);
          tma_store_3d(tm_lo, t + 2 * kTileHalf, 64 * p, y, z);
          if (REV) tma_store_3d(tm_dv, t + 4 * kTileHalf, 64 * p, y, z);
        }
        tma_store_commit();
      }
    }
    if (warp == 20 && lane == 0) tma_store_wait_all();
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

// grid 2 B H: the heads forwards, then the heads backwards
template <int DKP>
__global__ void __launch_bounds__(NT, 1)
    delta_sweep_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_rh,
                       const __grid_constant__ CUtensorMap tm_rl,
                       const __grid_constant__ CUtensorMap tm_uh,
                       const __grid_constant__ CUtensorMap tm_ul,
                       const __grid_constant__ CUtensorMap tm_dv,
                       const __grid_constant__ CUtensorMap tm_sh,
                       const __grid_constant__ CUtensorMap tm_sl,
                       const __grid_constant__ CUtensorMap tm_dh,
                       const __grid_constant__ CUtensorMap tm_dl, const uint8_t *rec,
                       const float *__restrict__ S_init, const float *__restrict__ dS_final,
                       float *__restrict__ dS_init, Kept kept, int BH, int nch, int dv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  if (blockIdx.x < static_cast<unsigned>(BH)) {
    const Args a{rec, S_init, nullptr, kept.s_hi, kept.s_lo, nch, dv};
    run<DKP, false>(smem_raw, &tm_q, &tm_k, &tm_v, &tm_rh, &tm_rl, nullptr, &tm_sh, &tm_sl, a,
                    blockIdx.x);
  } else {
    const Args a{rec, dS_final, dS_init, kept.d_hi, kept.d_lo, nch, dv};
    run<DKP, true>(smem_raw, &tm_q, &tm_k, &tm_do, &tm_uh, &tm_ul, &tm_dv, &tm_dh, &tm_dl, a,
                   blockIdx.x - BH);
  }
}

}  // namespace sweep

// ------------------------------------------------------------------ grad
namespace grad {

// One CTA per chunk.  Warps 0-15 are the epilogues: lane quarter warp % 4, a
// quarter of the columns each; warp 16 loads and issues the products.  For
// <S0, D> the epilogue threads take S0 into registers before D replaces it.
// Rows 0-63 of every product are tokens of the key side (du, giving dk), rows
// 64-127 tokens of the query side (dO, giving dq):
//   T = [du; dO] r^T         W = [K; Q] K^T                 (N = C)
//   A = [du; dO] S0^T        B = [r; .] D^T                 (N = d_k)
//   F = [-(Y + Y^T), M^T; M, 0] [K; Q]                      (N = d_k, 2 C deep)
// T and W give M, Y, dbeta (the diagonal of du r^T) and E; then
//   dk = e^(gamma_C - gamma) beta B + F - e^gamma beta A    dq = e^gamma A + F
// du and r enter as pairs.  [du_lo; 0] takes a zero tile, so that its products
// add nothing to the query rows.
// S0 and D share a buffer (D is fetched once the product with S0 is done), and
// the left operand of F lies where [du; dO] was.
constexpr int NT = 544;
constexpr int kEpi = 512;
constexpr uint32_t kOffKQ = 0;                          // 2 panels: k over q
constexpr uint32_t kOffU = 2 * kPanelKQ;                // 2 panels: du hi over dO
constexpr uint32_t kOffUl = kOffU + 2 * kPanelKQ;       // 2 panels: du lo over zeros
constexpr uint32_t kOffR = kOffUl + 2 * kPanelKQ;       // 2 panels: r hi over r lo
constexpr uint32_t kOffS = kOffR + 2 * kPanelKQ;        // hi: 2 panels [d_v, 64]; lo
constexpr uint32_t kStateHalf = 2 * kPanelKQ;           // hi or lo of a state
constexpr uint32_t kOffF = kOffU;                       // F's left operand: hi 2 panels, lo 2 panels
constexpr uint32_t kOffScal = kOffS + 2 * kStateHalf;   // e^gamma, e^(gamma_C - gamma), beta, gamma..
constexpr uint32_t kOffRed = kOffScal + kScalBytes + kGamBytes;
// column sums of E [4][64], its row sums [4][2][64], what S0 hands on
// [4][2][64], what goes to D [4][64], <S0, D> [16]
constexpr uint32_t kRedFloats = 4 * C + 8 * C + 8 * C + 4 * C + 16;
constexpr uint32_t kOffBar = kOffRed + kRedFloats * 4;
constexpr uint32_t kSmemBytes = kOffBar + 96;
static_assert(kSmemBytes <= 232448, "exceeds the per-CTA shared memory of sm_100");

constexpr uint32_t kTmA = 0, kTmB = 128, kTmF = 256, kTmT = 384, kTmW = 448, kTmCols = 512;

struct Args {
  const uint8_t *rec;
  float *dg, *dbeta;
  int N, nch, dv;
};

template <int DKP>
__global__ void __launch_bounds__(NT, 1)
    delta_grad_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_do,
                      const __grid_constant__ CUtensorMap tm_rh,
                      const __grid_constant__ CUtensorMap tm_rl,
                      const __grid_constant__ CUtensorMap tm_uh,
                      const __grid_constant__ CUtensorMap tm_ul,
                      const __grid_constant__ CUtensorMap tm_sh,
                      const __grid_constant__ CUtensorMap tm_sl,
                      const __grid_constant__ CUtensorMap tm_dh,
                      const __grid_constant__ CUtensorMap tm_dl,
                      const __grid_constant__ CUtensorMap tm_dq,
                      const __grid_constant__ CUtensorMap tm_dk, const Args a) {
  constexpr int DK = 64 * DKP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sm = smem_raw;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (sb & 1023u) {
    if (tid == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  const long head = blockIdx.x / a.nch;
  const int c = static_cast<int>(blockIdx.x % a.nch), z = static_cast<int>(head);
  const int plane = static_cast<int>(blockIdx.x);
  const int n0 = c * C, n = min(C, a.N - n0), vp = a.dv / 64;
  // loaded: inputs, S0, D; done: T and W, A, all; S0 is read, F's operand written
  const uint32_t b_in = sb + kOffBar, b_s = b_in + 8, b_d = b_in + 16, b_tw = b_in + 24,
                 b_a = b_in + 32, b_f = b_in + 40, b_read = b_in + 48, b_op = b_in + 56;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + 64);
  float *scal = reinterpret_cast<float *>(sm + kOffScal);
  const float *eg = scal, *el = scal + C, *be = scal + 2 * C, *gh = scal + kScalBytes / 4,
              *gl = gh + C, *colf = gl + C, *e0 = colf + C, *e1 = e0 + C;
  float *red = reinterpret_cast<float *>(sm + kOffRed);
  float *r_col = red, *r_row = red + 4 * C, *r_a = r_row + 8 * C, *r_b = r_a + 8 * C,
        *r_sd = r_b + 4 * C;

  auto load_state = [&](const CUtensorMap *hi, const CUtensorMap *lo, uint32_t full) {
    mbar_arrive_expect_tx(full, 2 * DKP * vp * kTileHalf);
    for (int p = 0; p < DKP; ++p)
      for (int v = 0; v < vp; ++v) {
        const uint32_t t = sb + kOffS + p * kPanelKQ + v * kTileHalf;
        tma_load_3d(t, hi, full, 64 * p, 64 * v, plane);
        tma_load_3d(t + kStateHalf, lo, full, 64 * p, 64 * v, plane);
      }
  };
  if (tid == kEpi) {
    for (int i = 0; i < 6; ++i) mbar_init(b_in + 8 * i, 1);
    mbar_init(b_read, kEpi / 32);
    mbar_init(b_op, kEpi / 32);
    fence_mbar_init();
    grid_dependency_wait();   // the sweeps
    mbar_arrive_expect_tx(b_in, (2 * DKP + 5 * vp) * kTileHalf + kScalBytes + kGamBytes);
    for (int p = 0; p < DKP; ++p) {
      tma_load_3d(sb + kOffKQ + p * kPanelKQ, &tm_k, b_in, 64 * p, n0, z);
      tma_load_3d(sb + kOffKQ + p * kPanelKQ + kTileHalf, &tm_q, b_in, 64 * p, n0, z);
    }
    for (int p = 0; p < vp; ++p) {
      const uint32_t o = p * kPanelKQ;
      tma_load_3d(sb + kOffU + o, &tm_uh, b_in, 64 * p, n0, z);
      tma_load_3d(sb + kOffU + o + kTileHalf, &tm_do, b_in, 64 * p, n0, z);
      tma_load_3d(sb + kOffUl + o, &tm_ul, b_in, 64 * p, n0, z);
      tma_load_3d(sb + kOffR + o, &tm_rh, b_in, 64 * p, n0, z);
      tma_load_3d(sb + kOffR + o + kTileHalf, &tm_rl, b_in, 64 * p, n0, z);
    }
    bulk_load(sb + kOffScal, a.rec + static_cast<long>(plane) * kRecord + kRecScal,
              kScalBytes + kGamBytes, b_in);
    load_state(&tm_sh, &tm_sl, b_s);
  }
  for (uint32_t i = tid * 16; i < 2 * kTileHalf; i += NT * 16)   // [du_lo; 0]
    *reinterpret_cast<uint4 *>(sm + kOffUl + (i / kTileHalf) * kPanelKQ + kTileHalf + i % kTileHalf) =
        make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const uint64_t dKQ = sdesc_sw128(sb + kOffKQ, 16, 1024);
  const uint64_t dKQmn = sdesc_sw128(sb + kOffKQ, kPanelKQ, 1024);
  const uint64_t dU = sdesc_sw128(sb + kOffU, 16, 1024), dUl = sdesc_sw128(sb + kOffUl, 16, 1024);
  const uint64_t dR = sdesc_sw128(sb + kOffR, 16, 1024);
  const uint64_t dS = sdesc_sw128(sb + kOffS, kPanelKQ, 1024);   // [d_v, d_k]: MN-major
  const uint64_t dF = sdesc_sw128(sb + kOffF, 16, 1024);
  constexpr uint32_t idC = idesc_bf16(128, C, 0, 0), idK = idesc_bf16(128, DK, 0, 1);
  auto kstep = [](int ks) -> uint64_t { return ((ks >> 2) * kPanelKQ + (ks & 3) * 32) >> 4; };
  // D (+)= A (rows of d_v) by a state, both terms of it or hi alone
  auto by_state = [&](uint32_t d, uint64_t A, int terms, bool add) {
    for (int term = 0; term < terms; ++term)
      for (int ks = 0; ks < 4 * vp; ++ks)
        umma_bf16(tmem + d, A + kstep(ks), dS + ((term * kStateHalf + ks * 2048) >> 4), idK,
                  add || term + ks > 0);
  };
  // a wait that runs out leaves wrong values behind, and the error flag
  if (warp == kEpi / 32) {
    if (lane == 0) {
      bool ok = mbar_wait(b_in, 0);
      tc_fence_after();
      if (ok) {
        for (int term = 0; term < 3; ++term)
          for (int ks = 0; ks < 4 * vp; ++ks)
            umma_bf16(tmem + kTmT, (term == 2 ? dUl : dU) + kstep(ks),
                      dR + (term == 1 ? kTileHalf >> 4 : 0) + kstep(ks), idC, term + ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4 * DKP; ++ks)
          umma_bf16(tmem + kTmW, dKQ + kstep(ks), dKQ + kstep(ks), idC, ks > 0);
      }
      umma_commit(b_tw);
      ok = mbar_wait(b_s, 0) && ok;
      tc_fence_after();
      if (ok) {
        by_state(kTmA, dU, 2, false);
        by_state(kTmA, dUl, 1, true);
      }
      umma_commit(b_a);
      const bool read = mbar_wait(b_read, 0), done = mbar_wait(b_a, 0);
      ok = read && done && ok;
      const bool second = ok;
      if (ok) {
        load_state(&tm_dh, &tm_dl, b_d);
        ok = mbar_wait(b_d, 0);
        tc_fence_after();
      }
      if (ok) {
        by_state(kTmB, dR, 2, false);
        by_state(kTmB, dR + (kTileHalf >> 4), 1, true);
      }
      ok = mbar_wait(b_op, 0) && ok;
      tc_fence_after();
      if (ok)
        for (int term = 0; term < 2; ++term)
          for (int ks = 0; ks < 8; ++ks)
            umma_bf16(tmem + kTmF, dF + ((term * 2 * kPanelKQ) >> 4) + kstep(ks),
                      dKQmn + ((ks * 2048) >> 4), idK, term + ks > 0);
      umma_commit(b_f);
      mbar_wait(b_f, 0);
      if (!ok) {   // the loads have to land before the CTA exits
        mbar_wait(b_in, 0);
        mbar_wait(b_s, 0);
        if (second) mbar_wait(b_d, 0);
      }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    return;
  }
  mbar_wait(b_in, 0);

  // row t of the key side (rows 0-63) or the query side, columns s0 .. s0 + 15
  const int row = (warp & 3) * 32 + lane, t = row & 63, b16 = warp >> 2, s0 = 16 * b16;
  const bool qside = (warp & 3) >= 2;
  const uint32_t lf = static_cast<uint32_t>((warp & 3) * 32) << 16;
  // each thread the same 16-byte pieces of S0's and of D's tiles
  constexpr int kPieces = 2 * DKP;
  uint4 sh[kPieces], sl[kPieces];
  auto piece = [&](int i) {
    const uint32_t idx = tid + i * kEpi;   // 512 pieces a tile of 64 rows
    return kOffS + ((idx >> 9) / vp) * kPanelKQ + ((idx >> 9) % vp) * kTileHalf + (idx & 511) * 16;
  };
  mbar_wait(b_s, 0);
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (i < DKP * vp) {
      sh[i] = *reinterpret_cast<const uint4 *>(sm + piece(i));
      sl[i] = *reinterpret_cast<const uint4 *>(sm + piece(i) + kStateHalf);
    }
  __syncwarp();
  if (lane == 0) mbar_arrive(b_read);

  mbar_wait(b_tw, 0);
  tc_fence_after();
  float mv[16];   // Y or M of this thread's row and columns
  {
    uint32_t tv[16], wv[16];
    tmem_ld<16>(tmem + lf + kTmT + s0, tv);
    tmem_ld<16>(tmem + lf + kTmW + s0, wv);
    tmem_wait_ld();
    const float bt = qside ? 1.f : be[t], ht = gh[t], lt = gl[t];
    const int rb = t >> 4;
    float rsum = 0.f, dbeta = 0.f, g[16];
    // Gam as in prep.  Masks are factors, not branches: an expf under a branch
    // of its own cost 170 cycles an element here, 43 without
    const float rf =
        (b16 < rb ? 1.f : 0.f) * expf(b16 < rb ? (ht - gh[s0 + 15]) + (lt - gl[s0 + 15]) : 0.f);
    const float on_diag = b16 == rb ? 1.f : 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(colf + s0 + i);
      g[i] = rf * f.x; g[i + 1] = rf * f.y; g[i + 2] = rf * f.z; g[i + 3] = rf * f.w;
    }
    const bool diag = (b16 >> 1) == (warp & 1);   // some of these rows have the block on it
    if (diag) {
      if (fabsf(gh[s0] - gh[s0 + 15]) < kMildGates) {
        const float f0 = on_diag * e0[t];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e4 = *reinterpret_cast<const float4 *>(e1 + s0 + i);
          const float es[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) g[i + x] += s0 + i + x <= t ? f0 * es[x] : 0.f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float in = s0 + i <= t ? on_diag : 0.f;
          g[i] += in * expf(in > 0.f ? (ht - gh[s0 + i]) + (lt - gl[s0 + i]) : 0.f);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)   // of du r^T
        dbeta = s0 + i == t ? __uint_as_float(tv[i]) : dbeta;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 b4 = *reinterpret_cast<const float4 *>(be + s0 + i);
      const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int s = s0 + i + x;
        float m = g[i + x] * bt * bs[x] * __uint_as_float(tv[i + x]);
        if (!qside && s >= t) m = 0.f;
        mv[i + x] = m;
        float ev = s < t ? m * __uint_as_float(wv[i + x]) : 0.f;
        ev = qside ? ev : -ev;
        wv[i + x] = __float_as_uint(ev);
        rsum += ev;
      }
    }
    if (!qside && b16 == rb && t < n) a.dbeta[head * a.N + n0 + t] = dbeta;
    r_row[b16 * 2 * C + (qside ? C : 0) + t] = rsum;
    // column sums over this warp's 32 rows: eight at a time, halving the
    // values and the lanes that share them
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float e[8], x4[4], x2[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = __uint_as_float(wv[8 * j + i]);
      const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float send = h16 ? e[i] : e[4 + i];
        x4[i] = (h16 ? e[4 + i] : e[i]) + __shfl_xor_sync(0xffffffffu, send, 16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float send = h8 ? x4[i] : x4[2 + i];
        x2[i] = (h8 ? x4[2 + i] : x4[i]) + __shfl_xor_sync(0xffffffffu, send, 8);
      }
      float x = (h4 ? x2[1] : x2[0]) + __shfl_xor_sync(0xffffffffu, h4 ? x2[0] : x2[1], 4);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      const int at = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
      if ((lane & 3) == 0) r_col[(warp & 3) * C + s0 + 8 * j + at] = x;
    }
  }
  // the products of du and dO are done: F's operand in their place
  mbar_wait(b_a, 0);
  uint8_t *fh = sm + kOffF, *fl = fh + 2 * kPanelKQ;
  // an element of F's left operand: panel = column / 64
  auto f_at = [](int r, int col) -> uint32_t {
    return (col >> 6) * kPanelKQ + sw128_offset(r, (col & 63) * 2);
  };
  {
    // row t: -Y (key rows), M (query rows), in the columns of K; zeros in the
    // query rows' columns of Q
    const int r = qside ? C + t : t;
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      uint32_t h[4], l[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = make_float2(mv[i + 2 * x], mv[i + 2 * x + 1]);
        split2(qside ? f : make_float2(-f.x, -f.y), h[x], l[x]);
      }
      const uint32_t o = f_at(r, s0 + i);
      *reinterpret_cast<uint4 *>(fh + o) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4 *>(fl + o) = make_uint4(l[0], l[1], l[2], l[3]);
      if (qside) {
        const uint32_t oz = f_at(r, C + s0 + i);
        *reinterpret_cast<uint4 *>(fh + oz) = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(fl + oz) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  named_bar_sync(1, kEpi);
  // transposed: -Y^T above the diagonal, M^T beside it
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int s = s0 + i;
    const float f = qside ? mv[i] : -mv[i];
    const __nv_bfloat16 h = __float2bfloat16_rn(f);
    const __nv_bfloat16 l = __float2bfloat16_rn(f - __bfloat162float(h));
    const uint32_t o = f_at(s, qside ? C + t : t);
    if (qside || s < t) {
      *reinterpret_cast<__nv_bfloat16 *>(fh + o) = h;
      *reinterpret_cast<__nv_bfloat16 *>(fl + o) = l;
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(b_op);
  mbar_wait(b_d, 0);
  {
    float sd = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (i < DKP * vp) {
        const uint4 dh = *reinterpret_cast<const uint4 *>(sm + piece(i));
        const uint4 dl = *reinterpret_cast<const uint4 *>(sm + piece(i) + kStateHalf);
        const uint32_t a1[4] = {sh[i].x, sh[i].y, sh[i].z, sh[i].w};
        const uint32_t a2[4] = {sl[i].x, sl[i].y, sl[i].z, sl[i].w};
        const uint32_t b1[4] = {dh.x, dh.y, dh.z, dh.w}, b2[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sd = fmaf(lo_f32(a1[x]) + lo_f32(a2[x]), lo_f32(b1[x]) + lo_f32(b2[x]), sd);
          sd = fmaf(hi_f32(a1[x]) + hi_f32(a2[x]), hi_f32(b1[x]) + hi_f32(b2[x]), sd);
        }
      }
    sd = warp_sum(sd);
    if (lane == 0) r_sd[warp] = sd;
  }
  mbar_wait(b_f, 0);
  tc_fence_after();

  // dk (key rows) and dq: columns of d_k by quarters
  {
    const float f1 = qside ? eg[t] : -eg[t] * be[t], f2 = el[t] * be[t];
    const uint8_t *own = sm + kOffKQ + (qside ? kTileHalf : 0);
    float sa = 0.f, sbb = 0.f;
#pragma unroll 1
    for (int j = b16 * (DK / 4); j < (b16 + 1) * (DK / 4); j += 16) {
      uint32_t va[16], vb[16], vf[16];
      tmem_ld<16>(tmem + lf + kTmA + j, va);
      tmem_ld<16>(tmem + lf + kTmF + j, vf);
      if (!qside) tmem_ld<16>(tmem + lf + kTmB + j, vb);
      tmem_wait_ld();
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; i += 8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(
            own + ((j + i) >> 6) * kPanelKQ + sw128_offset(t, ((j + i) & 63) * 2));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const float kq = y & 1 ? hi_f32(ww[y >> 1]) : lo_f32(ww[y >> 1]);
          const float pa = f1 * __uint_as_float(va[i + y]);
          sa = fmaf(kq, pa, sa);
          float pb = 0.f;
          if (!qside) {
            pb = f2 * __uint_as_float(vb[i + y]);
            sbb = fmaf(kq, pb, sbb);
          }
          x[i + y] = pa + pb + __uint_as_float(vf[i + y]);
        }
      }
      // where r was, which every product has read
      uint32_t p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = pack2(x[2 * i], x[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<uint4 *>(sm + kOffR + (j >> 6) * kPanelKQ +
                                   sw128_offset(row, (j & 63) * 2 + 16 * i)) =
            make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
    }
    r_a[b16 * 2 * C + row] = sa;
    if (!qside) r_b[b16 * C + t] = sbb;
  }
  tc_fence_before();
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {   // rows past the last token are left out
    for (int p = 0; p < DKP; ++p) {
      tma_store_3d(&tm_dk, sb + kOffR + p * kPanelKQ, 64 * p, n0, z);
      tma_store_3d(&tm_dq, sb + kOffR + p * kPanelKQ + kTileHalf, 64 * p, n0, z);
    }
    tma_store_commit();
    tma_store_wait_read();
  }
  if (a.dg && warp == 1) {
    // suffix sums of (row sums - column sums of E + what S0 hands on), and
    // exclusive prefix sums of what goes to D, over 64 tokens: two a lane
    float suf[2], pre[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int x = 2 * lane + i;
      float v = 0.f, w = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) v += r_row[q * C + x] + r_a[q * C + x];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v -= r_col[q * C + x];
        w += r_b[q * C + x];
      }
      suf[i] = v;
      pre[i] = w;
    }
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kEpi / 32; ++w) all += r_sd[w];
    float S = suf[0] + suf[1], P = pre[0] + pre[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_down_sync(0xffffffffu, S, o);
      const float y = __shfl_up_sync(0xffffffffu, P, o);
      if (lane + o < 32) S += x;
      if (lane >= o) P += y;
    }
    float before = __shfl_up_sync(0xffffffffu, P, 1);
    if (lane == 0) before = 0.f;
    const float tail = eg[C - 1] * all;
    const long at = head * a.N + n0 + 2 * lane;
    if (2 * lane < n) a.dg[at] = S + before + tail;
    if (2 * lane + 1 < n) a.dg[at + 1] = (S - suf[0]) + (before + pre[0]) + tail;
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

}  // namespace grad
}  // namespace delta
}  // namespace linattn
