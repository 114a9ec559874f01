// The gated delta rule on the 5th-generation tensor cores: bf16 with d_k and
// d_v in {64, 128}, chunks of C = 64 tokens.
//
// Inside a chunk, with S0 the state before it, gamma the running sums of the
// gates, Gam_ts = exp(gamma_t - gamma_s), N = strictly lower (Gam o K K^T) and
// P = lower (Gam o Q K^T), the recurrence is a unit triangular solve:
//   X = V - e^gamma K S0,   (I + N diag(beta)) r = X,   u = beta r
//   O = e^gamma Q S0 + P u,   S <- e^gamma_C S0 + K^T (e^(gamma_C - gamma) u).
// The solve is done once per chunk and head, away from the chain of chunks:
// (I + N diag(beta))^-1 = I + G diag(beta) with G strictly lower, so that
//   r = X + G (beta X)
// is a product.  G serves the reverse recurrence as well: with dU the gradient
// that reaches u from the chunk's outputs and its last state,
//   du = dU + G^T (beta dU).
//
// Kernels:
//   prep   every chunk of every head at once: G, P and the chunk's scalars
//   chain  one CTA per head, or per segment of a head, walks its chunks: X, r, O,
//          S; or S alone, from a given state and from the unit matrix, whose end
//          is the segment's transition
//   carry  joins the segments: the state each one starts from
//
// Precision.  An fp32 operand of a matrix product (S, beta X, u, G, P) enters
// as a pair of bf16 values, hi = bf16(x) and lo = bf16(x - hi), 16 bits of it;
// lo x lo products are left out.  k, q and v are bf16 already and enter as they
// are; decays multiply fp32 accumulators, never an operand that was exact.
// With single bf16 operands the state was off by 2e-3 after 1024 tokens, with
// pairs by 3e-6 to 4e-6, and d beta and dg by up to 7e-6 (fp32 arithmetic: 2e-7 to
// 4e-7; that is what the CUDA cores give); the pair costs two instructions where
// the other operand is exact and three where both are pairs.  A third word would
// cost half as many again, and the 512 columns of TMEM hold none.
#pragma once
#include "common.cuh"
#include "delta_simt.cuh"
#include "sm100.cuh"

namespace linattn {
namespace delta {

constexpr int C = 64;                            // tokens per chunk
constexpr uint32_t kTileHalf = 8192;             // 64 rows x 128 bytes (64 bf16)
constexpr uint32_t kPanelKQ = 2 * kTileHalf;     // per 64 columns: 64 rows of k, then 64 of q

// What prep leaves for a chunk: images of shared-memory tiles (rows of 128
// bytes, 16-byte pieces swizzled), fetched whole by bulk copies.
constexpr uint32_t kRecG = 0;                    // G hi, G lo
constexpr uint32_t kRecP = 2 * kTileHalf;        // P hi, P lo
constexpr uint32_t kRecScal = 4 * kTileHalf;     // e^gamma, e^(gamma_C - gamma), beta: 3 x 64 fp32
constexpr int kRest = 3 * C;                     // and what the rounding of e^gamma_C left out
constexpr uint32_t kScalBytes = (kRest + 4) * 4;
// behind them: gamma (high, low), e^(gamma_b - gamma) to the last token b of 16,
// e^(gamma - gamma_a) and e^(gamma_a - gamma) from the first, a
constexpr uint32_t kGamBytes = 5 * C * 4;
constexpr uint32_t kRecord = 4 * kTileHalf + 3 * 1024;
static_assert(kRecScal + kScalBytes + kGamBytes <= kRecord, "a record holds the scalars");
// The state takes e^gamma_C with that rest: the rounding is the same 2^-25 in every
// chunk of one slow gate, and adds up over them.
// A block of 16 tokens whose gates sum to less than this takes its decays as
// e^(gamma_t - gamma_a) e^(gamma_a - gamma_s), the second factor at most e^60;
// others (a new document inside) as exponentials of the differences.  The fp32
// exponents of the two factors round to 2^-19 at most, and do so only between
// tokens far from a: 1e-7 of S and out with any gates (simulated), below the pairs.
constexpr float kMildGates = 60.f;

// hi and lo bf16 pairs of two fp32 values (a in the low half)
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo) {
  hi = pack2(x.x, x.y);
  const float2 r = ffma2(make_float2(lo_f32(hi), hi_f32(hi)), make_float2(-1.f, -1.f), x);
  lo = pack2(r.x, r.y);
}
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  split2(make_float2(a, b), hi, lo);
}
// x - hi of a packed pair, rounded and packed
__device__ __forceinline__ uint32_t lo_pair(float2 x, uint32_t hi) {
  const float2 r = ffma2(make_float2(lo_f32(hi), hi_f32(hi)), make_float2(-1.f, -1.f), x);
  return pack2(r.x, r.y);
}
__device__ __forceinline__ float2 as_f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}
// a - b, pairwise
__device__ __forceinline__ float2 fsub2(float2 a, float2 b) {
  return ffma2(b, make_float2(-1.f, -1.f), a);
}

// fp32 values times the decay of a chunk, by its scalars (kRest)
template <int NC>
__device__ __forceinline__ void scale_state(uint32_t (&v)[NC], const float *scal) {
  const float2 f = make_float2(scal[C - 1], scal[C - 1]), rest = make_float2(scal[kRest], scal[kRest]);
#pragma unroll
  for (int i = 0; i < NC; i += 2) {
    const float2 x = as_f2(v[i], v[i + 1]), y = ffma2(x, f, fmul2(x, rest));
    v[i] = __float_as_uint(y.x);
    v[i + 1] = __float_as_uint(y.y);
  }
}

// 1-D bulk copy shared -> global (sizes and addresses multiples of 16 bytes).
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}

// The loads and stores of sm100.cuh by their number of columns.
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[NC]) {
  if constexpr (NC == 32) tmem_ld_32x32b_x32(taddr, r);
  else tmem_ld_32x32b_x16(taddr, r);
}
template <int NC>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[NC]) {
  if constexpr (NC == 32) tmem_st_32x32b_x32(taddr, r);
  else if constexpr (NC == 16) tmem_st_32x32b_x16(taddr, r);
  else tmem_st_32x32b_x8(taddr, r);
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d (16 x 8, fp32) += a (16 x 16) b (16 x 8), bf16 operands in one warp's registers
__device__ __forceinline__ void mma_16816(float *d, const uint32_t *a, const uint32_t *b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// A 16 x 16 block of fp32 values in one warp, as the accumulators of two
// 16 x 8 products lay them out: v[0..3] columns 0-7, v[4..7] columns 8-15; lane
// (g, t) = (lane / 4, lane % 4) holds rows g and g + 8, columns 2 t and 2 t + 1.
struct Block16 {
  float v[8];
};
// The same block as the left operand of a 16-deep product: the accumulator
// layout is that operand's layout, pair by pair.
struct Left16 {
  uint32_t hi[4], lo[4];
};
__device__ __forceinline__ Left16 left_of(const Block16 &b) {
  Left16 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) split2(b.v[2 * i], b.v[2 * i + 1], a.hi[i], a.lo[i]);
  return a;
}
// acc += a b for a right operand given as ldmatrix_x4_trans fragments of its
// hi and lo parts (fragments 0, 1: columns 0-7; 2, 3: columns 8-15)
__device__ __forceinline__ void mma_block(Block16 &acc, const Left16 &a, const uint32_t (&bh)[4],
                                          const uint32_t (&bl)[4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    mma_16816(acc.v + 4 * n, a.hi, bh + 2 * n);
    mma_16816(acc.v + 4 * n, a.hi, bl + 2 * n);
    mma_16816(acc.v + 4 * n, a.lo, bh + 2 * n);
  }
}

// Pairs of C tokens: hi of 16 tokens (one step of a product) in 8 columns,
// then their lo in 8.
__device__ __forceinline__ uint32_t pair_col(int ks, bool lo) { return 16u * ks + (lo ? 8u : 0u); }

// D (+)= pairs(A) pairs(B) over C tokens: hi hi, hi lo, lo hi
// (a tile of 64 x 64 and its lo behind it; MN: contracted over its rows)
template <bool MN>
__device__ __forceinline__ void pairs_hi(uint32_t tmem, uint32_t d, uint32_t a, uint64_t b,
                                         bool add) {
  constexpr uint32_t id = idesc_bf16(128, C, 0, MN ? 1 : 0);
#pragma unroll
  for (int term = 0; term < 2; ++term)
#pragma unroll
    for (int ks = 0; ks < C / 16; ++ks)
      umma_bf16_ts(tmem + d, tmem + a + pair_col(ks, false),
                   b + (term == 1 ? kTileHalf >> 4 : 0) + ((ks * (MN ? 2048 : 32)) >> 4), id,
                   add || term + ks > 0);
}
template <bool MN>
__device__ __forceinline__ void pairs_lo(uint32_t tmem, uint32_t d, uint32_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16(128, C, 0, MN ? 1 : 0);
#pragma unroll
  for (int ks = 0; ks < C / 16; ++ks)
    umma_bf16_ts(tmem + d, tmem + a + pair_col(ks, true), b + ((ks * (MN ? 2048 : 32)) >> 4), id, 1u);
}

// ------------------------------------------------------------------ prep
namespace prep {

constexpr int NT = 128;
constexpr uint32_t kOffG = 0;                    // k, q tiles; then N, then G
constexpr uint32_t kOffP = 2 * kTileHalf;        //             then P
constexpr uint32_t kOffDiag = 4 * kTileHalf;     // diagonal blocks of N, transposed, fp32 [4][16][20]
constexpr uint32_t kDiagPitch = 20;              // rows start on 16 bytes
constexpr uint32_t kOffT = kOffDiag + 4 * 16 * kDiagPitch * 4;   // I + beta G_jj, hi and lo: 8 x [16][16]
constexpr uint32_t kOffScal = kOffT + 8 * 512;   // e^gamma, e^(gamma_C - gamma), beta, the rest
constexpr uint32_t kOffGam = kOffScal + kScalBytes;   // gamma hi, gamma lo, e^(gamma_b - gamma), ..
constexpr uint32_t kOffBar = kOffGam + kGamBytes;
constexpr uint32_t kSmemBytes = kOffBar + 64;

// One CTA per chunk, of the chunks c0 .. c0 + cnt - 1 of every head.  With
// `behind` the grid was launched to run beside the chain of the chunks before
// (it needs nothing of it); its last block then ends after that grid, so that
// what is ordered after this grid is ordered after both.
//
// A single product forms K K^T and Q K^T: the k rows over the q rows are one
// 128-row left operand, the k rows the right one.  Warps 0 and 1 get K K^T and
// write N, warps 2 and 3 write P.  Gam is a product of two exponentials taken
// per token: over the last token b of the column block off the diagonal,
// e^(gamma_t - gamma_b) e^(gamma_b - gamma_s), both at most 1, and over the
// first of the block on it (kMildGates; with exponentials of their own on the
// diagonal blocks 2048 chunks took 39.5 us, so 36.2).  gamma is summed in fp64
// and kept as two fp32 words, so that a difference of large sums is as exact as
// its parts.
//
// G = -(N + N beta G): the diagonal blocks by substitution, a lane to a column;
// then warp i has row block i to itself, from the diagonal to the left:
//   G_ij = -(N_ij + sum_{j < k <= i} G_ik beta_k N_kj) (I + beta_j G_jj).
// The left operands are the warp's own accumulators, so blocks pass from one
// product to the next in registers; 16 x 16 x 16 products are far below the
// tile of tcgen05, so these run as warp-level ones.
template <int DKP>
__global__ void __launch_bounds__(NT, 5) delta_prep_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                        const __grid_constant__ CUtensorMap tm_k,
                                                        const float *__restrict__ g,
                                                        const float *__restrict__ beta,
                                                        uint8_t *__restrict__ rec, int N, int nch,
                                                        int c0, int cnt, int behind) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sm = smem_raw;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (sb & 1023u) {
    if (tid == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  const long head = blockIdx.x / cnt;
  const int c = c0 + static_cast<int>(blockIdx.x % cnt);
  const int n0 = c * C, n = min(C, N - n0);
  const uint32_t bar_load = sb + kOffBar, bar_mma = bar_load + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + 16);
  float *eg = reinterpret_cast<float *>(sm + kOffScal), *el = eg + C, *sbeta = el + C;
  float *gh = reinterpret_cast<float *>(sm + kOffGam), *gl = gh + C, *colf = gl + C, *e0 = colf + C,
        *e1 = e0 + C;
  float *diag = reinterpret_cast<float *>(sm + kOffDiag);

  if (tid == 0) {
    mbar_init(bar_load, 1);
    mbar_init(bar_mma, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(bar_load, 2 * DKP * kTileHalf);
    for (int p = 0; p < DKP; ++p) {
      tma_load_3d(sb + p * kPanelKQ, &tm_k, bar_load, 64 * p, n0, static_cast<int>(head));
      tma_load_3d(sb + p * kPanelKQ + kTileHalf, &tm_q, bar_load, 64 * p, n0,
                  static_cast<int>(head));
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 64);
    tmem_relinquish();
  }
  if (warp == 1) {   // scalars: lane takes tokens lane and lane + 32
    const long tok = head * N + n0;
    double x[2];
    float b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane + 32 * i;
      x[i] = t < n && g ? static_cast<double>(gate_floor(g[tok + t])) : 0.0;
      b[i] = t < n ? beta[tok + t] : 0.f;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y0 = __shfl_up_sync(0xffffffffu, x[0], o);
      const double y1 = __shfl_up_sync(0xffffffffu, x[1], o);
      if (lane >= o) {
        x[0] += y0;
        x[1] += y1;
      }
    }
    x[1] += __shfl_sync(0xffffffffu, x[0], 31);
    const double last = __shfl_sync(0xffffffffu, x[1], 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = lane + 32 * i;
      const double blk = __shfl_sync(0xffffffffu, x[i], lane | 15);
      const double first = __shfl_sync(0xffffffffu, x[i], lane & 16);
      gh[t] = static_cast<float>(x[i]);
      gl[t] = static_cast<float>(x[i] - static_cast<double>(static_cast<float>(x[i])));
      eg[t] = expf(static_cast<float>(x[i]));
      el[t] = expf(static_cast<float>(last - x[i]));
      colf[t] = expf(static_cast<float>(blk - x[i]));
      e0[t] = expf(static_cast<float>(x[i] - first));
      e1[t] = expf(fminf(static_cast<float>(first - x[i]), 80.f));
      sbeta[t] = b[i];
      if (t == C - 1) {   // from a half on e^gamma_C - 1 is exact; less does not add up
        const float less = expm1f(static_cast<float>(last));
        *reinterpret_cast<float4 *>(eg + kRest) =
            make_float4(fabsf(less) < 0.5f ? less - (eg[t] - 1.f) : 0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // [K; Q] K^T
  bool ok = true;
  if (tid == 0) {
    ok = mbar_wait(bar_load, 0);
    if (ok) {
      constexpr uint32_t id = idesc_bf16(128, C, 0, 0);
      const uint64_t d = sdesc_sw128(sb, 16, 1024);
#pragma unroll
      for (int ks = 0; ks < 4 * DKP; ++ks) {
        const uint64_t o = ((ks >> 2) * kPanelKQ + (ks & 3) * 32) >> 4;
        umma_bf16(tmem, d + o, d + o, id, ks > 0);
      }
    }
    umma_commit(bar_mma);
  }
  __syncwarp();
  ok = mbar_wait(bar_mma, 0) && ok;
  tc_fence_after();

  // N (warps 0, 1) or P (warps 2, 3): row t, 16 columns at a time
  {
    const bool is_p = warp >= 2;
    const int t = (warp & 1) * 32 + lane, rb = t >> 4;
    uint8_t *tile = sm + (is_p ? kOffP : kOffG);
    uint32_t acc[2][32];
    tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(warp * 32) << 16), acc[0]);
    if (warp & 1) tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 32, acc[1]);
    tmem_wait_ld();
    __syncthreads();   // every warp has its accumulators (and the k, q tiles are read)
    const float ht = gh[t], lt = gl[t];
#pragma unroll
    for (int cb = 0; cb < 4; ++cb) {
      float w[16];
      if ((cb >> 1) <= (warp & 1)) {   // the others are above the diagonal
        const float rf = (cb < rb ? 1.f : 0.f) *
                         expf(cb < rb ? (ht - gh[16 * cb + 15]) + (lt - gl[16 * cb + 15]) : 0.f);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(colf + 16 * cb + i);
          w[i] = rf * f.x; w[i + 1] = rf * f.y; w[i + 2] = rf * f.z; w[i + 3] = rf * f.w;
        }
        if ((cb >> 1) == (warp & 1)) {   // some of these rows have it on the diagonal
          const float on_diag = cb == rb ? 1.f : 0.f;
          if (fabsf(gh[16 * cb] - gh[16 * cb + 15]) < kMildGates) {
            const float f = on_diag * e0[t];
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 e4 = *reinterpret_cast<const float4 *>(e1 + 16 * cb + i);
              const float es[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int s = 16 * cb + i + x;
                w[i + x] += s < t || (s == t && is_p) ? f * es[x] : 0.f;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int s = 16 * cb + i;
              const float in = s < t || (s == t && is_p) ? on_diag : 0.f;
              w[i] += in * expf(in > 0.f ? (ht - gh[s]) + (lt - gl[s]) : 0.f);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] *= __uint_as_float(acc[cb >> 1][(cb & 1) * 16 + i]);
        if (!is_p && cb == rb)
#pragma unroll
          for (int i = 0; i < 16; ++i) diag[(rb * 16 + i) * kDiagPitch + (t & 15)] = w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 0.f;
      }
      uint32_t h[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split2(w[2 * i], w[2 * i + 1], h[i], l[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t o = sw128_offset(t, cb * 32 + i * 16);
        *reinterpret_cast<uint4 *>(tile + o) =
            make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        *reinterpret_cast<uint4 *>(tile + kTileHalf + o) =
            make_uint4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
      }
    }
  }
  __syncthreads();

  // diagonal block `warp` of G, column j: x_i = -(N_ij + sum_{j<k<i} N_ik beta_k x_k),
  // each x_k added to all later rows as soon as it is known: one
  // multiply-add stands between an x and the next, and the columns of N can
  // be fetched ahead of them
  {
    const int j = lane & 15;
    const float *nt = diag + warp * 16 * kDiagPitch;
    float x[16], y[16];   // sums, then G; beta_k x_k
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(nt + j * kDiagPitch + i);
      x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;   // 0 for i <= j
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      x[k] = k > j ? -x[k] : 0.f;
      y[k] = sbeta[16 * warp + k] * x[k];
#pragma unroll
      for (int i = (k + 1) / 4 * 4; i < 16; i += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(nt + k * kDiagPitch + i);
        if (i > k) x[i] = fmaf(f.x, y[k], x[i]);
        if (i + 1 > k) x[i + 1] = fmaf(f.y, y[k], x[i + 1]);
        if (i + 2 > k) x[i + 2] = fmaf(f.z, y[k], x[i + 2]);
        if (i + 3 > k) x[i + 3] = fmaf(f.w, y[k], x[i + 3]);
      }
    }
    // G_jj into the tile (lanes 0-15: hi, 16-31: lo), I + beta G_jj beside it
    const bool low = lane >= 16;
    __nv_bfloat16 *tj = reinterpret_cast<__nv_bfloat16 *>(sm + kOffT + warp * 1024 + (low ? 512 : 0));
    uint8_t *tile = sm + kOffG + (low ? kTileHalf : 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float e = y[i] + (i == j ? 1.f : 0.f);
      const __nv_bfloat16 eh = __float2bfloat16_rn(e), xh = __float2bfloat16_rn(x[i]);
      tj[i * 16 + j] = low ? __float2bfloat16_rn(e - __bfloat162float(eh)) : eh;
      *reinterpret_cast<__nv_bfloat16 *>(
          tile + sw128_offset(16 * warp + i, (16 * warp + j) * 2)) =
          low ? __float2bfloat16_rn(x[i] - __bfloat162float(xh)) : xh;
    }
  }
  __syncthreads();

  // row block `warp`, from the diagonal to the left
  Block16 out[3];
  {
    const int gq = lane >> 2, tq = lane & 3;
    Left16 left[3];        // G_{i, i-d} beta, d = 0..2
    auto beta_left = [&](const Block16 &b, int blk) {
      Block16 s;
      const float *bb = sbeta + 16 * blk + 2 * tq;
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s.v[4 * nb + e] = b.v[4 * nb + e] * bb[8 * nb + (e & 1)];
      return left_of(s);
    };
    // block (bi, bj) of the tile in the accumulator layout
    auto block_at = [&](int bi, int bj) {
      Block16 b;
#pragma unroll
      for (int nb = 0; nb < 2; ++nb)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t o = sw128_offset(16 * bi + gq + 8 * r, (16 * bj + 8 * nb + 2 * tq) * 2);
          const uint32_t h = *reinterpret_cast<const uint32_t *>(sm + kOffG + o);
          const uint32_t l = *reinterpret_cast<const uint32_t *>(sm + kOffG + kTileHalf + o);
          b.v[4 * nb + 2 * r] = lo_f32(h) + lo_f32(l);
          b.v[4 * nb + 2 * r + 1] = hi_f32(h) + hi_f32(l);
        }
      return b;
    };
    left[0] = beta_left(block_at(warp, warp), warp);
    const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lch = lane >> 4;
#pragma unroll
    for (int dj = 1; dj < 4; ++dj) {
      const int j = warp - dj;
      if (j >= 0) {
        Block16 z = block_at(warp, j);
#pragma unroll
        for (int d = 0; d < dj; ++d) {
          uint32_t bh[4], bl[4];
          const uint32_t o = sb + kOffG + sw128_offset(16 * (warp - d) + lrow, (2 * j + lch) * 16);
          ldmatrix_x4_trans(o, bh);
          ldmatrix_x4_trans(o + kTileHalf, bl);
          mma_block(z, left[d], bh, bl);
        }
        uint32_t th[4], tl[4];
        const uint32_t o = sb + kOffT + j * 1024 + lrow * 32 + lch * 16;
        ldmatrix_x4_trans(o, th);
        ldmatrix_x4_trans(o + 512, tl);
        Block16 r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          z.v[e] = -z.v[e];
          r.v[e] = 0.f;
        }
        mma_block(r, left_of(z), th, tl);
        out[dj - 1] = r;
        if (dj < 3) left[dj] = beta_left(r, j);
      }
    }
  }
  __syncthreads();   // every warp has read the blocks of N it needs
  {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int dj = 1; dj < 4; ++dj) {
      const int j = warp - dj;
      if (j >= 0)
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t h, l;
            split2(out[dj - 1].v[4 * nb + 2 * r], out[dj - 1].v[4 * nb + 2 * r + 1], h, l);
            const uint32_t o =
                sw128_offset(16 * warp + gq + 8 * r, (16 * j + 8 * nb + 2 * tq) * 2);
            *reinterpret_cast<uint32_t *>(sm + kOffG + o) = h;
            *reinterpret_cast<uint32_t *>(sm + kOffG + kTileHalf + o) = l;
          }
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    uint8_t *dst = rec + (head * nch + c) * kRecord;
    if (ok) {
      bulk_store(dst, sb, 4 * kTileHalf);
      bulk_store(dst + kRecScal, sb + kOffScal, kScalBytes + kGamBytes);
    }
    tma_store_commit();
    tma_store_wait_read();
    if (!ok) mbar_wait(bar_load, 0);   // the loads have to land before the CTA exits
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
  if (behind && blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}

}  // namespace prep

// ------------------------------------------------------------------ chain
namespace chain {

// Everything is held transposed, a TMEM lane to a column of S (d_v <= 128):
// S^T [d_v, d_k], X^T, r^T and O^T [d_v, C].  So every product has M = 128,
// its left operand (S, beta X, u) comes out of the epilogue of the product
// before in the same lanes and goes back to TMEM as the A operand without
// passing through shared memory, and its right operand (k, q, G, P) is a tile
// as it was loaded.  Decays and beta are factors of a token: of a column here,
// broadcast from shared memory.
//
// Warps: 0 loads, 1 issues the products of the chain, 2 those that only the
// outputs wait for, 4-19 the chain (lane quarter warp % 4, a quarter of the
// columns each), 20-23 the outputs; 3 idles.  24 warps leave a thread 80
// registers: with d_k = 128 a chain warp's 32 columns of S and what goes on beside
// them spill 196 bytes a thread.
constexpr int NT = 768;
constexpr uint32_t kOffKQ = 0;                    // 2 panels: k over q (stage 0), q over k (stage 1)
constexpr uint32_t kOffV = 2 * kPanelKQ;          // 2 panels of 64 rows
constexpr uint32_t kOffRec = kOffV + 2 * kTileHalf;   // G, P, scalars
constexpr uint32_t kStage = kOffRec + kRecord;
static_assert(kStage % 1024 == 0, "tiles start on 1024 bytes");
constexpr int kStages = 2;
constexpr uint32_t kOffOut = kStages * kStage;     // out: 2 panels of 64 rows
constexpr uint32_t kOffEye = kOffOut + 2 * kTileHalf;   // the 64 x 64 identity
constexpr uint32_t kOffBar = kOffEye + kTileHalf;
constexpr uint32_t kSmemBytes = kOffBar + 256;
static_assert(kSmemBytes <= 232448, "exceeds the per-CTA shared memory of sm_100");

enum Bar {
  kFull0 = 0, kFull1, kFullP0, kFullP1,   // k, q, v, G and the scalars are loaded; P is
  kFree0, kFree1, kFreeP0, kFreeP1,   // k, q, v, G are read; P is
  kKQ, kGX, kS, kO,                   // a product is done (once a chunk)
  // the chain warps' operands are in TMEM, hi before lo: the products by hi
  // run while the warps make lo
  kXhReady, kXlReady, kUhReady, kUlReady, kShReady, kSlReady, kUReady,
  kOScaled0, kOScaled1, kFinal, kFinalO, kNumBars
};
static_assert(kNumBars * 8 <= 224, "barrier area overflow");
constexpr uint32_t kOffTmem = 224;

// TMEM columns
constexpr uint32_t kTmS = 0;      // S^T, fp32 (d_k columns)
constexpr uint32_t kTmSh = 128;   // S^T hi (d_k / 2 columns)
constexpr uint32_t kTmSl = 192;   // S^T lo
constexpr uint32_t kTmO0 = 256;   // O^T of the odd chunks
constexpr uint32_t kTmX = 320;    // S^T k^T; then the pairs of beta X; then of u
constexpr uint32_t kTmO1 = 384;   // O^T of the even chunks
constexpr uint32_t kTmG = 448;    // V^T + (beta X)^T G^T; then the pairs of e^(gamma_C - gamma) u
constexpr uint32_t kTmCols = 512;

// A grid walks chunks c0 .. c0 + len segs - 1 of `all` (the last segment may be
// shorter), a CTA per head and segment.
//   STATE = false: with the outputs.  Segment 0 starts from S_init, segment j
//     from slot j - 1 of carry, the last one writes S_final.  S_init and S_final
//     may be one buffer: a CTA reads its head's state before the first chunk
//     and writes it behind the last.
//   STATE = true: what a segment does to a state, S -> M S + B, without
//     outputs.  B of segments 0 .. segs - 2 (segment 0's from S_init) goes to the
//     slots of carry, M of segments 1 .. segs - 2 to those of trans, transposed.
//     M is the chain with v = 0 that starts from the identity: d_k columns in the
//     place of d_v.
struct Args {
  const uint8_t *rec;
  const float *S_init;
  float *carry, *trans, *S_final;
  int all, c0, len, segs, BH, dv;
};

template <int DKP, bool STATE>
__global__ void __launch_bounds__(NT, 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_out, const Args args) {
  constexpr int DK = 64 * DKP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sm = smem_raw;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31;
  // the same in every lane, and known to be: roles branch without divergence
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (sb & 1023u) {
    if (tid == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  grid_launch_dependents();   // the next slab's prep may start beside this grid
  const int unit = blockIdx.x / args.BH;
  const long head = blockIdx.x % args.BH;
  const bool trans = STATE && unit >= args.segs - 1;
  const int seg = trans ? unit - (args.segs - 2) : unit;
  const int all = args.all, c0 = args.c0 + seg * args.len, nch = min(args.len, all - c0);
  const int dv = trans ? DK : args.dv;
  const uint8_t *rec = args.rec;
  const long state = static_cast<long>(DK) * args.dv;
  const float *S_in = seg == 0 ? (args.S_init ? args.S_init + head * state : nullptr)
                      : STATE  ? nullptr
                               : args.carry + (static_cast<long>(seg - 1) * args.BH + head) * state;
  float *S_out = STATE ? args.carry + (static_cast<long>(seg) * args.BH + head) * state
                 : seg == args.segs - 1 && args.S_final ? args.S_final + head * state
                                                        : nullptr;
  auto bar = [&](int i) { return sb + kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + kOffTmem);

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const int n = i >= kXhReady && i <= kUReady ? 16 : i == kOScaled0 || i == kOScaled1 ? 4 : 1;
      mbar_init(bar(i), n);
    }
    fence_mbar_init();
  }
  // the identity; and zeros where v has no second panel
  for (int i = tid; i < C * C / 2; i += NT) {
    const uint32_t r = i / (C / 2), e = 2 * (i % (C / 2));
    *reinterpret_cast<uint32_t *>(sm + kOffEye + sw128_offset(r, e * 2)) =
        r == e ? 0x00003f80u : r == e + 1 ? 0x3f800000u : 0u;
  }
  if (dv == 64 || trans)
    for (int s = 0; s < kStages; ++s)
      for (uint32_t i = tid * 16 + (trans ? 0 : kTileHalf); i < 2 * kTileHalf; i += NT * 16)
        *reinterpret_cast<uint4 *>(sm + s * kStage + kOffV + i) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();   // prep, or the states between the segments
  // A wait that runs out sets the error word.  It ends a role of one lane; warps
  // that work as a whole, or meet at a named barrier, go through all their
  // chunks without waiting again: a lane that left could leave the others
  // waiting for it without a limit.
  auto wait = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity & 1); };
  bool ok = true;
  auto pass = [&](int i, uint32_t parity) {
    if (ok) ok = wait(i, parity);
    tc_fence_after();
  };

  if (warp == 0) {
    if (lane == 0) {
      const int vp = trans ? 0 : dv / 64;
      int issued = 0, issued_p = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        const uint32_t st = sb + s * kStage;
        const int y = (c0 + c) * C, z = static_cast<int>(head);
        const uint8_t *r = rec + (head * all + c0 + c) * kRecord;
        // the scalars beside G are read until the output of the stage's last
        // chunk is scaled
        if (c >= kStages && (!wait(kFree0 + s, (c >> 1) + 1) ||
                             (!STATE && !wait(kOScaled0 + s, (c >> 1) + 1))))
          break;
        const uint32_t full = bar(kFull0 + s);
        mbar_arrive_expect_tx(full, ((STATE ? 1 : 2) * DKP + vp + 2) * kTileHalf + kScalBytes);
        for (int p = 0; p < DKP; ++p) {
          const uint32_t t = st + kOffKQ + p * kPanelKQ;
          tma_load_3d(t + (!STATE && s ? kTileHalf : 0), &tm_k, full, 64 * p, y, z);
          if (!STATE) tma_load_3d(t + (s ? 0 : kTileHalf), &tm_q, full, 64 * p, y, z);
        }
        for (int p = 0; p < vp; ++p)
          tma_load_3d(st + kOffV + p * kTileHalf, &tm_v, full, 64 * p, y, z);
        bulk_load(st + kOffRec + kRecScal, r + kRecScal, kScalBytes, full);
        bulk_load(st + kOffRec + kRecG, r + kRecG, 2 * kTileHalf, full);
        issued = c + 1;
        if (STATE) continue;
        if (c >= kStages && !wait(kFreeP0 + s, (c >> 1) + 1)) break;
        mbar_arrive_expect_tx(bar(kFullP0 + s), 2 * kTileHalf);
        bulk_load(st + kOffRec + kRecP, r + kRecP, 2 * kTileHalf, bar(kFullP0 + s));
        issued_p = c + 1;
      }
      // the copies this thread started have to land before the CTA exits
      for (int c = issued - kStages < 0 ? 0 : issued - kStages; c < issued; ++c) {
        mbar_wait(bar(kFull0 + (c & 1)), (c >> 1) & 1);
        if (c < issued_p) mbar_wait(bar(kFullP0 + (c & 1)), (c >> 1) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idKQ = idesc_bf16(128, STATE ? C : 2 * C, 0, 0);   // k and q: K-major
      constexpr uint32_t idK = idesc_bf16(128, DK, 0, 1);    // k as [C, d_k]: MN-major, N = d_k
      const uint64_t dKQ = sdesc_sw128(sb + kOffKQ, 16, 1024);
      const uint64_t dKmn = sdesc_sw128(sb + kOffKQ, kPanelKQ, 1024);
      const uint64_t dG = sdesc_sw128(sb + kOffRec + kRecG, 16, 1024);
      constexpr uint32_t idV = idesc_bf16(128, C, 1, 0);        // v as [C, d_v]: MN-major
      const uint64_t dV = sdesc_sw128(sb + kOffV, kTileHalf, 1024);
      const uint64_t dEye = sdesc_sw128(sb + kOffEye, 16, 1024);
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        const uint32_t ph = c >> 1;
        const uint64_t so = static_cast<uint64_t>(s) * (kStage >> 4);
        // V^T through the identity, exactly: the transposed v comes out of TMEM
        // far sooner than element by element out of shared memory, which the
        // products keep busy
        if (!wait(kFull0 + s, ph)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks)
          umma_bf16(tmem + kTmG, dV + so + ((ks * 2048) >> 4), dEye + ((ks * 32) >> 4), idV, ks > 0);
        // S^T [k; q]^T: X and O side by side.  An instruction with N = 128
        // takes hardly longer to issue than one with N = 64, and issuing them
        // is what the chain waits for; O has two places, left and right of X
        // (the outputs' product of the chunk before has read u, and began only
        // after the output warps were done with this chunk's place of O)
        if (!STATE && c >= 1 && !wait(kO, c - 1)) break;
        bool in = true;
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          if (!(in = in && wait(term ? kSlReady : kShReady, c))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4 * DKP; ++ks)
            umma_bf16_ts(tmem + (!STATE && s ? kTmO0 : kTmX), tmem + (term ? kTmSl : kTmSh) + 8 * ks,
                         dKQ + so + (((ks >> 2) * kPanelKQ + (ks & 3) * 32) >> 4), idKQ,
                         term + ks > 0);
        }
        if (!in) break;
        umma_commit(bar(kKQ));
        if (!wait(kXhReady, c)) break;
        tc_fence_after();
        pairs_hi<false>(tmem, kTmG, kTmX, dG + so, true);
        if (!wait(kXlReady, c)) break;
        tc_fence_after();
        pairs_lo<false>(tmem, kTmG, kTmX, dG + so);
        umma_commit(bar(kGX));
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          if (!(in = in && wait(term ? kUlReady : kUhReady, c))) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            umma_bf16_ts(tmem + kTmS, tmem + kTmG + pair_col(ks, term),
                         dKmn + so + (((!STATE && s ? kTileHalf : 0) + ks * 2048) >> 4), idK, 1u);
        }
        if (!in) break;
        umma_commit(bar(kS));
        umma_commit(bar(kFree0 + s));
      }
      umma_commit(bar(kFinal));
      mbar_wait(bar(kFinal), 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    if (!STATE && lane == 0) {
      // O += u P^T, beside the state's product and the pairs of S
      const uint64_t dP = sdesc_sw128(sb + kOffRec + kRecP, 16, 1024);
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        if (!wait(kFullP0 + s, c >> 1) || !wait(kOScaled0 + s, c >> 1) || !wait(kUReady, c)) break;
        tc_fence_after();
        const uint64_t p = dP + static_cast<uint64_t>(s) * (kStage >> 4);
        pairs_hi<false>(tmem, s ? kTmO0 : kTmO1, kTmX, p, true);
        pairs_lo<false>(tmem, s ? kTmO0 : kTmO1, kTmX, p);
        umma_commit(bar(kO));
        umma_commit(bar(kFreeP0 + s));
      }
      umma_commit(bar(kFinalO));
      mbar_wait(bar(kFinalO), 0);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 20) {
    const int wq = warp & 3, h = (warp - 4) >> 2;
    const int col = wq * 32 + lane;                     // column of S
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    constexpr int SC = DK / 4;                          // d_k columns per warp
    const int k0 = h * SC;
    const int t0 = 16 * h;                              // first token of this warp
    auto arrive = [&](int i) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    auto scal = [&](int c) {
      return reinterpret_cast<const float *>(sm + (c & 1) * kStage + kOffRec + kRecScal);
    };
    // the pairs of this warp's columns of S
    auto put_pairs = [&](const uint32_t (&v)[SC]) {
#pragma unroll
      for (int j = 0; j < SC; j += 16) {
        uint32_t hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          hi[i] = pack2(__uint_as_float(v[j + 2 * i]), __uint_as_float(v[j + 2 * i + 1]));
        tmem_st<8>(tmem + lf + kTmSh + (k0 + j) / 2, hi);
      }
      arrive(kShReady);
#pragma unroll
      for (int j = 0; j < SC; j += 16) {
        uint32_t lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = as_f2(v[j + 2 * i], v[j + 2 * i + 1]);
          lo[i] = lo_pair(f, pack2(f.x, f.y));
        }
        tmem_st<8>(tmem + lf + kTmSl + (k0 + j) / 2, lo);
      }
      arrive(kSlReady);
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
        v[i] = trans          ? (k0 + i == col ? __float_as_uint(1.f) : 0u)
               : S_in && live ? __float_as_uint(S_in[static_cast<long>(k0 + i) * dv + col])
                              : 0u;
      put_pairs(v);
      put_scaled(v, scal(0));
    }
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const float *eg = scal(c) + t0, *el = eg + C, *be = el + C;
      float2 x[8];   // e^gamma S^T k, then r
      pass(kKQ, c);
      {
        uint32_t d[16], v[16], p[8];
        tmem_ld<16>(tmem + lf + kTmX + t0, d);
        tmem_ld<16>(tmem + lf + kTmG + t0, v);
        tmem_wait_ld();
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e = *reinterpret_cast<const float4 *>(eg + i);
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          x[i / 2] = fmul2(make_float2(e.x, e.y), as_f2(d[i], d[i + 1]));
          x[i / 2 + 1] = fmul2(make_float2(e.z, e.w), as_f2(d[i + 2], d[i + 3]));
          y[i / 2] = fmul2(make_float2(b.x, b.y), fsub2(as_f2(v[i], v[i + 1]), x[i / 2]));
          y[i / 2 + 1] =
              fmul2(make_float2(b.z, b.w), fsub2(as_f2(v[i + 2], v[i + 3]), x[i / 2 + 1]));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pack2(y[i].x, y[i].y);
        tmem_st<8>(tmem + lf + kTmX + t0, p);
        arrive(kXhReady);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = lo_pair(y[i], p[i]);
        tmem_st<8>(tmem + lf + kTmX + t0 + 8, p);
      }
      arrive(kXlReady);
      pass(kGX, c);
      {
        // first what the state waits for, e^(gamma_C - gamma) u; then u
        uint32_t d[16], p[8];
        tmem_ld<16>(tmem + lf + kTmG + t0, d);
        tmem_wait_ld();
        float2 y[8];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          const float4 e = *reinterpret_cast<const float4 *>(el + i);
          x[i / 2] = fmul2(make_float2(b.x, b.y), fsub2(as_f2(d[i], d[i + 1]), x[i / 2]));
          x[i / 2 + 1] =
              fmul2(make_float2(b.z, b.w), fsub2(as_f2(d[i + 2], d[i + 3]), x[i / 2 + 1]));
          y[i / 2] = fmul2(make_float2(e.x, e.y), x[i / 2]);
          y[i / 2 + 1] = fmul2(make_float2(e.z, e.w), x[i / 2 + 1]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = pack2(y[i].x, y[i].y);
        tmem_st<8>(tmem + lf + kTmG + t0, p);
        arrive(kUhReady);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = lo_pair(y[i], p[i]);
        tmem_st<8>(tmem + lf + kTmG + t0 + 8, p);
      }
      arrive(kUlReady);
      if constexpr (!STATE) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2(x[i], p[i], p[8 + i]);
        tmem_st<16>(tmem + lf + kTmX + t0, p);
        arrive(kUReady);
      }
      pass(kS, c);
      uint32_t v[SC];
      tmem_ld<SC>(tmem + lf + kTmS + k0, v);
      tmem_wait_ld();
      if (c + 1 < nch) {
        put_pairs(v);
        // S times the next chunk's decay, before that chunk's product adds to
        // it (that product waits for kUhReady, behind these stores)
        pass(kFull0 + (s ^ 1), (c + 1) >> 1);
        put_scaled(v, scal(c + 1));
      } else if (trans) {
        if (live) {
          float4 *dst = reinterpret_cast<float4 *>(
              args.trans + ((static_cast<long>(seg - 1) * args.BH + head) * DK + col) * DK + k0);
#pragma unroll
          for (int i = 0; i < SC; i += 4)
            dst[i / 4] = make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]),
                                     __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
        }
      } else if (S_out && live) {
#pragma unroll
        for (int i = 0; i < SC; ++i)
          S_out[static_cast<long>(k0 + i) * dv + col] = __uint_as_float(v[i]);
      }
    }
    tc_fence_before();
  } else if (!STATE && warp >= 20) {
    const int wq = warp & 3;
    const int col = wq * 32 + lane;
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    uint8_t *ot = sm + kOffOut + (col >> 6) * kTileHalf + (col & 7) * 2;
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (((col & 63) >> 3) ^ i) << 4;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const uint32_t tO = tmem + lf + (s ? kTmO0 : kTmO1);
      pass(kFull0 + s, c >> 1);
      pass(kKQ, c);
      const float *eg = reinterpret_cast<const float *>(sm + s * kStage + kOffRec + kRecScal);
#pragma unroll 1
      for (int b = 0; b < C; b += 16) {
        uint32_t d[16];
        tmem_ld<16>(tO + b, d);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 e = *reinterpret_cast<const float4 *>(eg + b + i);
          d[i] = __float_as_uint(__uint_as_float(d[i]) * e.x);
          d[i + 1] = __float_as_uint(__uint_as_float(d[i + 1]) * e.y);
          d[i + 2] = __float_as_uint(__uint_as_float(d[i + 2]) * e.z);
          d[i + 3] = __float_as_uint(__uint_as_float(d[i + 3]) * e.w);
        }
        tmem_st<16>(tO + b, d);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOScaled0 + s));
      pass(kO, c);
      // transposed through shared memory: a lane writes its column, the bulk
      // store takes the rows (and leaves out those past the last token)
      if (warp == 20 && lane == 0) tma_store_wait_read();
      named_bar_sync(1, 128);
#pragma unroll
      for (int b = 0; b < C; b += 32) {
        uint32_t d[32];
        tmem_ld<32>(tO + b, d);
        tmem_wait_ld();
        if (live)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint32_t w = pack2(__uint_as_float(d[i]), __uint_as_float(d[i + 1]));
            *reinterpret_cast<uint16_t *>(ot + (b + i) * 128 + o[i & 7]) = static_cast<uint16_t>(w);
            *reinterpret_cast<uint16_t *>(ot + (b + i + 1) * 128 + o[(i + 1) & 7]) =
                static_cast<uint16_t>(w >> 16);
          }
      }
      tc_fence_before();   // before the next chunk's kOScaled, which lets go of this place of O
      fence_proxy_async_smem();
      named_bar_sync(1, 128);
      if (ok && warp == 20 && lane == 0) {
        for (int p = 0; p < dv / 64; ++p)
          tma_store_3d(&tm_out, sb + kOffOut + p * kTileHalf, 64 * p, (c0 + c) * C,
                       static_cast<int>(head));
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

// The states at the start of segments 2 .. segs - 1, in place of B in carry:
//   S_{j+1} = M_j S_j + B_j,   S_1 = B_0.
// Columns of S are independent: a block takes 16 of a head's, a thread a row, 8
// of them and a quarter of the inner index.  M lies transposed, so that
// threads read consecutive rows; the next M is in registers before this step's
// sums are joined, since the chain of steps is what the kernel waits for (one
// step of d_k = 128: 13.5 us with a thread to the whole inner index, 11.1 so;
// four of d_k = 64: 22.8 and 6.6).
constexpr int kCarryParts = 4;
template <int DK>
__global__ void __launch_bounds__(2 * kCarryParts * DK)
    delta_carry_kernel(float *carry, const float *trans, int segs, int BH,
                       int dv) {
  constexpr int KP = DK / kCarryParts;
  __shared__ __align__(16) float S[DK][16], part[kCarryParts][DK][17];
  const int r = threadIdx.x % DK, half = (threadIdx.x / DK) & 1, kp = threadIdx.x / (2 * DK);
  const int j0 = 8 * half, col = 16 * blockIdx.y;
  const long head = blockIdx.x, state = static_cast<long>(DK) * dv;
  grid_dependency_wait();
  auto fetch = [&](int j, float (&m)[KP]) {
    const float *M = trans + ((static_cast<long>(j - 1) * BH + head) * DK + kp * KP) * DK + r;
#pragma unroll
    for (int k = 0; k < KP; ++k) m[k] = j < segs - 1 ? M[k * DK] : 0.f;
  };
  // outputs: one element a thread and pass
  constexpr int OUT = DK * 16 / (2 * kCarryParts * DK);
  auto element = [&](int i) { return threadIdx.x + i * 2 * kCarryParts * DK; };
  float m[KP], b[OUT];
  fetch(1, m);
#pragma unroll
  for (int i = 0; i < OUT; ++i) {
    const int e = element(i);
    S[e / 16][e % 16] = carry[head * state + static_cast<long>(e / 16) * dv + col + e % 16];
  }
  for (int j = 1; j < segs - 1; ++j) {
    float *slot = carry + (static_cast<long>(j) * BH + head) * state + col;
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
      const int e = element(i);
      b[i] = slot[static_cast<long>(e / 16) * dv + e % 16];
    }
    __syncthreads();
    float x[8] = {};
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      const float4 p = *reinterpret_cast<const float4 *>(&S[kp * KP + k][j0]);
      const float4 q = *reinterpret_cast<const float4 *>(&S[kp * KP + k][j0 + 4]);
      x[0] = fmaf(m[k], p.x, x[0]); x[1] = fmaf(m[k], p.y, x[1]);
      x[2] = fmaf(m[k], p.z, x[2]); x[3] = fmaf(m[k], p.w, x[3]);
      x[4] = fmaf(m[k], q.x, x[4]); x[5] = fmaf(m[k], q.y, x[5]);
      x[6] = fmaf(m[k], q.z, x[6]); x[7] = fmaf(m[k], q.w, x[7]);
    }
    fetch(j + 1, m);
#pragma unroll
    for (int e = 0; e < 8; ++e) part[kp][r][j0 + e] = x[e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
      const int e = element(i);
      float v = b[i];
#pragma unroll
      for (int p = 0; p < kCarryParts; ++p) v += part[p][e / 16][e % 16];
      S[e / 16][e % 16] = v;
      slot[static_cast<long>(e / 16) * dv + e % 16] = v;
    }
  }
}

}  // namespace chain
}  // namespace delta
}  // namespace linattn
