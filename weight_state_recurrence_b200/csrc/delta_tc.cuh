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
// Two kernels:
//   prep   every chunk of every head at once: G, P and the chunk's scalars
//   chain  one CTA per head walks its chunks: X, r, O, S
//
// Precision.  An fp32 operand of a matrix product (S, beta X, u, G, P) enters
// as a pair of bf16 values, hi = bf16(x) and lo = bf16(x - hi), 16 bits of it;
// lo x lo products are left out.  k, q and v are bf16 already and enter as they
// are; decays multiply fp32 accumulators, never an operand that was exact.
// With single bf16 operands the state was off by 2e-3 after 1024 tokens, with
// pairs by 3e-6 (fp32 simulation: 2e-7); the pair costs two instructions where
// the other operand is exact and three where both are pairs.
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
constexpr uint32_t kScalBytes = 3 * C * 4;
constexpr uint32_t kRecord = 4 * kTileHalf + 1024;

// hi and lo bf16 pairs of two fp32 values (a in the low half)
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  hi = pack2(a, b);
  lo = pack2(a - lo_f32(hi), b - hi_f32(hi));
}

// 1-D bulk copy shared -> global (sizes and addresses multiples of 16 bytes).
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
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

// ------------------------------------------------------------------ prep
namespace prep {

constexpr int NT = 128;
constexpr uint32_t kOffG = 0;                    // k, q tiles; then N, then G
constexpr uint32_t kOffP = 2 * kTileHalf;        //             then P
constexpr uint32_t kOffDiag = 4 * kTileHalf;     // diagonal blocks of N, fp32 [4][16][20]
constexpr uint32_t kDiagPitch = 20;              // rows start on 16 bytes
constexpr uint32_t kOffT = kOffDiag + 4 * 16 * kDiagPitch * 4;   // I + beta G_jj, hi and lo: 8 x [16][16]
constexpr uint32_t kOffScal = kOffT + 8 * 512;   // e^gamma, e^(gamma_C - gamma), beta
constexpr uint32_t kOffGam = kOffScal + kScalBytes;   // gamma hi, gamma lo, e^(gamma_b - gamma)
constexpr uint32_t kOffBar = kOffGam + 3 * C * 4;
constexpr uint32_t kSmemBytes = kOffBar + 64;

// One CTA per chunk.  A single product forms K K^T and Q K^T: the k rows over
// the q rows are one 128-row left operand, the k rows the right one.  Warps 0
// and 1 get K K^T and write N, warps 2 and 3 write P.  Gam takes exponentials
// on the 16 x 16 diagonal blocks only; elsewhere it is the product
// e^(gamma_t - gamma_b) e^(gamma_b - gamma_s) over the last token b of the
// column block, both factors at most 1.  gamma is summed in fp64 and kept as
// two fp32 words, so that a difference of large sums is as exact as its parts.
//
// G = -(N + N beta G): the diagonal blocks by substitution, a lane to a column;
// then warp i has row block i to itself, from the diagonal to the left:
//   G_ij = -(N_ij + sum_{j < k <= i} G_ik beta_k N_kj) (I + beta_j G_jj).
// The left operands are the warp's own accumulators, so blocks pass from one
// product to the next in registers; 16 x 16 x 16 products are far below the
// tile of tcgen05, so these run as warp-level ones.
template <int DKP>
__global__ void __launch_bounds__(NT) delta_prep_kernel(const __grid_constant__ CUtensorMap tm_q,
                                                        const __grid_constant__ CUtensorMap tm_k,
                                                        const float *__restrict__ g,
                                                        const float *__restrict__ beta,
                                                        uint8_t *__restrict__ rec, int N, int nch) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sm = smem_raw;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sb & 1023u) {
    if (tid == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  const long head = blockIdx.x / nch;
  const int c = static_cast<int>(blockIdx.x % nch);
  const int n0 = c * C, n = min(C, N - n0);
  const uint32_t bar_load = sb + kOffBar, bar_mma = bar_load + 8;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + 16);
  float *eg = reinterpret_cast<float *>(sm + kOffScal), *el = eg + C, *sbeta = el + C;
  float *gh = reinterpret_cast<float *>(sm + kOffGam), *gl = gh + C, *colf = gl + C;
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
      x[i] = t < n && g ? static_cast<double>(fmaxf(g[tok + t], kGateFloor)) : 0.0;
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
      gh[t] = static_cast<float>(x[i]);
      gl[t] = static_cast<float>(x[i] - static_cast<double>(static_cast<float>(x[i])));
      eg[t] = expf(static_cast<float>(x[i]));
      el[t] = expf(static_cast<float>(last - x[i]));
      colf[t] = expf(static_cast<float>(blk - x[i]));
      sbeta[t] = b[i];
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
      if (cb < rb) {
        const float rf = expf((ht - gh[16 * cb + 15]) + (lt - gl[16 * cb + 15]));
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = rf * colf[16 * cb + i] * __uint_as_float(acc[cb >> 1][(cb & 1) * 16 + i]);
      } else if (cb == rb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 16 * cb + i;
          const float a = __uint_as_float(acc[cb >> 1][(cb & 1) * 16 + i]);
          const float d = expf(fminf((ht - gh[s]) + (lt - gl[s]), 0.f));
          w[i] = s < t ? d * a : (s == t && is_p ? a : 0.f);
        }
        if (!is_p)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(diag + (rb * 16 + (t & 15)) * kDiagPitch + 4 * i) =
                make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
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

  // diagonal block `warp` of G, column j: x_i = -(N_ij + sum_{j<k<i} N_ik beta_k x_k)
  {
    const int j = lane & 15;
    const float *nb = diag + warp * 16 * kDiagPitch;
    float y[16];   // beta_k x_k
    float x[16];
    x[0] = y[0] = 0.f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      float row[16];
#pragma unroll
      for (int m = 0; m < (i + 3) / 4; ++m) {
        const float4 f = *reinterpret_cast<const float4 *>(nb + i * kDiagPitch + 4 * m);
        row[4 * m] = f.x; row[4 * m + 1] = f.y; row[4 * m + 2] = f.z; row[4 * m + 3] = f.w;
      }
      float s0 = nb[i * kDiagPitch + j], s1 = 0.f;   // 0 for j >= i
#pragma unroll
      for (int k = 0; k < i; ++k) {
        if (k & 1) s1 = fmaf(row[k], y[k], s1);
        else s0 = fmaf(row[k], y[k], s0);
      }
      x[i] = i > j ? -(s0 + s1) : 0.f;
      y[i] = sbeta[16 * warp + i] * x[i];
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
    uint8_t *dst = rec + static_cast<long>(blockIdx.x) * kRecord;
    if (ok) {
      bulk_store(dst, sb, 4 * kTileHalf);
      bulk_store(dst + kRecScal, sb + kOffScal, kScalBytes);
    }
    tma_store_commit();
    tma_store_wait_read();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
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
// Warps: 0 loads, 1 issues the products, 4-11 the chain (lane quarter
// warp % 4, half of the columns each), 12-15 the outputs.
constexpr int NT = 512;
constexpr uint32_t kOffKQ = 0;                    // 2 panels: 64 rows of k over 64 of q
constexpr uint32_t kOffV = 2 * kPanelKQ;          // 2 panels of 64 rows
constexpr uint32_t kOffRec = kOffV + 2 * kTileHalf;   // G, P, scalars
constexpr uint32_t kStage = kOffRec + kRecord;
static_assert(kStage % 1024 == 0, "tiles start on 1024 bytes");
constexpr int kStages = 2;
constexpr uint32_t kOffBar = kStages * kStage;
constexpr uint32_t kSmemBytes = kOffBar + 256;
static_assert(kSmemBytes <= 232448, "exceeds the per-CTA shared memory of sm_100");

enum Bar {
  kFullKQ0 = 0, kFullKQ1, kFullV0, kFullV1, kFullR0, kFullR1, kFree0, kFree1,
  kKS, kQS, kGX, kS, kO,          // a product is done (once a chunk)
  kXReady, kUReady, kSReady,      // the chain warps' operands are in TMEM
  kOScaled, kOFree, kFinal, kNumBars
};
constexpr uint32_t kOffTmem = 200, kOffAbort = 204;

// TMEM columns
constexpr uint32_t kTmS = 0;      // S^T, fp32 (d_k columns)
constexpr uint32_t kTmSh = 128;   // S^T hi (d_k / 2 columns)
constexpr uint32_t kTmSl = 192;   // S^T lo
constexpr uint32_t kTmX = 256;    // S^T k^T; then the pairs of beta X; then of u
constexpr uint32_t kTmO = 320;    // O^T
constexpr uint32_t kTmG = 384;    // (beta X)^T G^T; then the pairs of e^(gamma_C - gamma) u
constexpr uint32_t kTmCols = 512;

// Pairs of C tokens: 32 tokens' hi in 16 columns, then their lo in 16.
__device__ __forceinline__ uint32_t pair_col(int ks, bool lo) {
  return 32u * (ks >> 1) + 8u * (ks & 1) + (lo ? 16u : 0u);
}

template <int DKP>
__global__ void __launch_bounds__(NT, 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const uint8_t *__restrict__ rec,
                       const float *__restrict__ S_init, __nv_bfloat16 *__restrict__ out,
                       float *__restrict__ S_final, int N, int nch, int dv) {
  constexpr int DK = 64 * DKP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *sm = smem_raw;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sb & 1023u) {
    if (tid == 0) atomicOr(&g_status, kStatusWaitTimeout);
    return;
  }
  const long head = blockIdx.x;
  auto bar = [&](int i) { return sb + kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + kOffBar + kOffTmem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + kOffBar + kOffAbort);

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      const int n = i == kXReady || i == kUReady || i == kSReady ? 8
                    : i == kOScaled || i == kOFree               ? 4 : 1;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // a wait that runs out ends the role; the others run out, or see the flag
  auto wait = [&](int i, uint32_t parity) {
    if (!*abort_flag && mbar_wait(bar(i), parity & 1)) return true;
    *abort_flag = 1;
    return false;
  };

  if (warp == 0) {
    if (lane == 0) {
      const int vp = dv / 64;
      int issued = 0;
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        if (c >= kStages && !wait(kFree0 + s, (c >> 1) + 1)) break;
        const uint32_t st = sb + s * kStage;
        const int y = c * C, z = static_cast<int>(head);
        const uint8_t *r = rec + (head * nch + c) * kRecord;
        mbar_arrive_expect_tx(bar(kFullKQ0 + s), 2 * DKP * kTileHalf);
        for (int p = 0; p < DKP; ++p) {
          tma_load_3d(st + kOffKQ + p * kPanelKQ, &tm_k, bar(kFullKQ0 + s), 64 * p, y, z);
          tma_load_3d(st + kOffKQ + p * kPanelKQ + kTileHalf, &tm_q, bar(kFullKQ0 + s), 64 * p, y, z);
        }
        mbar_arrive_expect_tx(bar(kFullR0 + s), 4 * kTileHalf + kScalBytes);
        bulk_load(st + kOffRec, r, 4 * kTileHalf, bar(kFullR0 + s));
        bulk_load(st + kOffRec + kRecScal, r + kRecScal, kScalBytes, bar(kFullR0 + s));
        mbar_arrive_expect_tx(bar(kFullV0 + s), vp * kTileHalf);
        for (int p = 0; p < vp; ++p)
          tma_load_3d(st + kOffV + p * kTileHalf, &tm_v, bar(kFullV0 + s), 64 * p, y, z);
        issued = c + 1;
      }
      // the copies this thread started have to land before the CTA exits
      for (int c = issued - kStages < 0 ? 0 : issued - kStages; c < issued; ++c)
        for (int b = kFullKQ0; b <= kFullR0; b += 2) mbar_wait(bar(b + (c & 1)), (c >> 1) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idC = idesc_bf16(128, C, 0, 0);     // k, q, G, P: K-major, N = C
      constexpr uint32_t idK = idesc_bf16(128, DK, 0, 1);    // k as [C, d_k]: MN-major, N = d_k
      const uint64_t dK = sdesc_sw128(sb + kOffKQ, 16, 1024);
      const uint64_t dKmn = sdesc_sw128(sb + kOffKQ, kPanelKQ, 1024);
      const uint64_t dG = sdesc_sw128(sb + kOffRec + kRecG, 16, 1024);
      const uint64_t dP = sdesc_sw128(sb + kOffRec + kRecP, 16, 1024);
      constexpr uint64_t kLo = kTileHalf >> 4;
      // D += pairs(A) B for an exact B (terms hi, lo) over C tokens or d_k
      auto state_by = [&](uint32_t d, uint64_t b) {
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < 4 * DKP; ++ks)
            umma_bf16_ts(tmem + d, tmem + (term ? kTmSl : kTmSh) + 8 * ks,
                         b + (((ks >> 2) * kPanelKQ + (ks & 3) * 32) >> 4), idC,
                         term + ks > 0);
      };
      // D (+)= pairs(A) pairs(B): hi hi, hi lo, lo hi
      auto pairs_by = [&](uint32_t d, uint32_t a, uint64_t b, bool add) {
#pragma unroll
        for (int term = 0; term < 3; ++term)
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            umma_bf16_ts(tmem + d, tmem + a + pair_col(ks, term == 2),
                         b + (term == 1 ? kLo : 0) + ((ks * 32) >> 4), idC,
                         add || term + ks > 0);
      };
      for (int c = 0; c < nch; ++c) {
        const int s = c & 1;
        const uint32_t ph = c >> 1;
        const uint64_t so = static_cast<uint64_t>(s) * (kStage >> 4);
        if (!wait(kFullKQ0 + s, ph) || !wait(kSReady, c)) break;
        tc_fence_after();
        state_by(kTmX, dK + so);
        umma_commit(bar(kKS));
        if (c > 0 && !wait(kOFree, c - 1)) break;
        tc_fence_after();
        state_by(kTmO, dK + so + (kTileHalf >> 4));
        umma_commit(bar(kQS));
        if (!wait(kFullR0 + s, ph) || !wait(kXReady, c)) break;
        tc_fence_after();
        pairs_by(kTmG, kTmX, dG + so, false);
        umma_commit(bar(kGX));
        if (!wait(kUReady, c)) break;
        tc_fence_after();
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < C / 16; ++ks)
            umma_bf16_ts(tmem + kTmS, tmem + kTmG + pair_col(ks, term),
                         dKmn + so + ((ks * 2048) >> 4), idK, 1u);
        umma_commit(bar(kS));
        if (!wait(kOScaled, c)) break;
        tc_fence_after();
        pairs_by(kTmO, kTmX, dP + so, true);
        umma_commit(bar(kO));
        umma_commit(bar(kFree0 + s));
      }
      umma_commit(bar(kFinal));
      mbar_wait(bar(kFinal), 0);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    const int wq = warp & 3, h = (warp - 4) >> 2;
    const int col = wq * 32 + lane;                     // column of S
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    constexpr int SB = DKP;                             // blocks of 32 d_k columns per warp
    const int k0 = h * 32 * SB;                         // first d_k column of this warp
    auto arrive = [&](int i) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(i));
    };
    auto scal = [&](int c) {
      return reinterpret_cast<const float *>(sm + (c & 1) * kStage + kOffRec + kRecScal);
    };
    // pairs of 32 columns k0 + 32 b .. of S, and S times the next chunk's decay
    auto put_pairs = [&](int b, const uint32_t (&v)[32]) {
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        split2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), hi[i], lo[i]);
      tmem_st_32x32b_x16(tmem + lf + kTmSh + (k0 + 32 * b) / 2, hi);
      tmem_st_32x32b_x16(tmem + lf + kTmSl + (k0 + 32 * b) / 2, lo);
    };
    auto put_scaled = [&](int b, uint32_t (&v)[32], float f) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
      tmem_st_32x32b_x32(tmem + lf + kTmS + k0 + 32 * b, v);
    };
    bool ok = wait(kFullR0, 0);
    if (ok) {
      const float f = scal(0)[C - 1];
#pragma unroll 1
      for (int b = 0; b < SB; ++b) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          v[i] = S_init && live
                     ? __float_as_uint(S_init[(head * DK + k0 + 32 * b + i) * dv + col])
                     : 0u;
        put_pairs(b, v);
        put_scaled(b, v, f);
      }
      arrive(kSReady);
    }
    for (int c = 0; ok && c < nch; ++c) {
      const int s = c & 1;
      const float *eg = scal(c) + 32 * h, *el = eg + C, *be = el + C;
      float x[32];
      // v of this lane's column, tokens 32 h ..
      if (!(ok = wait(kFullV0 + s, c >> 1))) break;
      {
        const uint8_t *vt = sm + s * kStage + kOffV + (col >> 6) * kTileHalf + 32 * h * 128 +
                            (col & 7) * 2;
        const uint32_t ch = (col & 63) >> 3;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          x[i] = live ? __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(
                                            vt + i * 128 + ((ch ^ (i & 7)) << 4)))
                                        << 16)
                      : 0.f;
      }
      if (!(ok = wait(kFullR0 + s, c >> 1) && wait(kKS, c))) break;
      tc_fence_after();
      {
        uint32_t d[32];
        tmem_ld_32x32b_x32(tmem + lf + kTmX + 32 * h, d);
        tmem_wait_ld();
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 e = *reinterpret_cast<const float4 *>(eg + i);
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          x[i] = fmaf(-e.x, __uint_as_float(d[i]), x[i]);
          x[i + 1] = fmaf(-e.y, __uint_as_float(d[i + 1]), x[i + 1]);
          x[i + 2] = fmaf(-e.z, __uint_as_float(d[i + 2]), x[i + 2]);
          x[i + 3] = fmaf(-e.w, __uint_as_float(d[i + 3]), x[i + 3]);
          split2(b.x * x[i], b.y * x[i + 1], p[i / 2], p[16 + i / 2]);
          split2(b.z * x[i + 2], b.w * x[i + 3], p[i / 2 + 1], p[16 + i / 2 + 1]);
        }
        tmem_st_32x32b_x32(tmem + lf + kTmX + 32 * h, p);
      }
      arrive(kXReady);
      if (!(ok = wait(kGX, c))) break;
      tc_fence_after();
      {
        uint32_t d[32];
        tmem_ld_32x32b_x32(tmem + lf + kTmG + 32 * h, d);
        tmem_wait_ld();
        uint32_t p[32], w[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(be + i);
          const float4 e = *reinterpret_cast<const float4 *>(el + i);
          const float u0 = b.x * (x[i] + __uint_as_float(d[i]));
          const float u1 = b.y * (x[i + 1] + __uint_as_float(d[i + 1]));
          const float u2 = b.z * (x[i + 2] + __uint_as_float(d[i + 2]));
          const float u3 = b.w * (x[i + 3] + __uint_as_float(d[i + 3]));
          split2(u0, u1, p[i / 2], p[16 + i / 2]);
          split2(u2, u3, p[i / 2 + 1], p[16 + i / 2 + 1]);
          split2(e.x * u0, e.y * u1, w[i / 2], w[16 + i / 2]);
          split2(e.z * u2, e.w * u3, w[i / 2 + 1], w[16 + i / 2 + 1]);
        }
        tmem_st_32x32b_x32(tmem + lf + kTmG + 32 * h, w);
        tmem_st_32x32b_x32(tmem + lf + kTmX + 32 * h, p);
      }
      arrive(kUReady);
      const bool last = c == nch - 1;
      if (!(ok = wait(kS, c))) break;
      tc_fence_after();
      if (!last) {
#pragma unroll 1
        for (int b = 0; b < SB; ++b) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + lf + kTmS + k0 + 32 * b, v);
          tmem_wait_ld();
          put_pairs(b, v);
        }
        arrive(kSReady);
        // S times the next chunk's decay, before that chunk's product adds to
        // it (that product waits for kUReady, behind these stores)
        if (!(ok = wait(kFullR0 + (s ^ 1), (c + 1) >> 1))) break;
        const float f = scal(c + 1)[C - 1];
#pragma unroll 1
        for (int b = 0; b < SB; ++b) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + lf + kTmS + k0 + 32 * b, v);
          tmem_wait_ld();
          put_scaled(b, v, f);
        }
      } else if (S_final) {
#pragma unroll 1
        for (int b = 0; b < SB; ++b) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(tmem + lf + kTmS + k0 + 32 * b, v);
          tmem_wait_ld();
          if (live)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              S_final[(head * DK + k0 + 32 * b + i) * dv + col] = __uint_as_float(v[i]);
        }
      }
    }
    tc_fence_before();
  } else if (warp >= 12) {
    const int wq = warp & 3;
    const int col = wq * 32 + lane;
    const bool live = wq * 32 < dv;
    const uint32_t lf = static_cast<uint32_t>(wq * 32) << 16;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      if (!wait(kFullR0 + s, c >> 1) || !wait(kQS, c)) break;
      tc_fence_after();
      const float *eg = reinterpret_cast<const float *>(sm + s * kStage + kOffRec + kRecScal);
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        uint32_t d[32];
        tmem_ld_32x32b_x32(tmem + lf + kTmO + 32 * b, d);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          d[i] = __float_as_uint(__uint_as_float(d[i]) * eg[32 * b + i]);
        tmem_st_32x32b_x32(tmem + lf + kTmO + 32 * b, d);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOScaled));
      if (!wait(kO, c)) break;
      tc_fence_after();
      uint32_t d[2][32];
      tmem_ld_32x32b_x32(tmem + lf + kTmO, d[0]);
      tmem_ld_32x32b_x32(tmem + lf + kTmO + 32, d[1]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kOFree));
      if (live) {
        // lanes 2 j and 2 j + 1 trade, so that each stores two columns of one
        // token: a warp's store covers 64 bytes of two tokens
        const int n = min(C, N - c * C), odd = lane & 1;
        __nv_bfloat16 *dst = out + (head * N + c * C + odd) * dv + (col & ~1);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float a = __uint_as_float(d[b][i]), e = __uint_as_float(d[b][i + 1]);
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : e, 1);
            const uint32_t w = odd ? pack2(got, e) : pack2(a, got);
            const int t = 32 * b + i;
            if (t + odd < n) *reinterpret_cast<uint32_t *>(dst + static_cast<long>(t) * dv) = w;
          }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmCols);
  }
}

}  // namespace chain
}  // namespace delta
}  // namespace linattn
