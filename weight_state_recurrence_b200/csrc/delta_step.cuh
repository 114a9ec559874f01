// One token of the gated delta rule for every head, the state updated in place:
//   r = v - a S^T k,  u = beta r,  S <- a S + k u^T,  out = S^T q,  a = exp(g).
// Bound by HBM traffic on the state (dk dv 4 bytes read and written per head).
// Built as decode.cuh is: one persistent CTA per SM, heads streamed through a
// ring of shared-memory stages by 1-D bulk copies, streaming 128-bit stores
// back.  The update needs S^T k before it can write anything, so the output is
// taken from the state before the update in the same pass,
//   out = a S^T q + (k . q) u,
// and a head costs one reduction over its rows instead of two.  A thread
// keeps its rows in registers between the two halves.
#pragma once
#include "common.cuh"
#include "decode.cuh"
#include "sm100.cuh"

namespace linattn {
namespace delta {

constexpr int kStepThreads = 256;
constexpr int kStepStages = 3;

template <int DK, int DV, typename T>
struct StepLayout {
  static constexpr uint32_t kS = DK * DV * 4;
  static constexpr uint32_t kQ = DK * sizeof(T);
  static constexpr uint32_t kV = DV * sizeof(T);
  static constexpr uint32_t kBytes = kS + 2 * kQ + kV;               // bulk bytes per head
  static constexpr uint32_t kStage = (kBytes + 127) / 128 * 128;
  static constexpr int TPR = DV / 4;                                  // threads per S row
  static constexpr int RPP = kStepThreads / TPR;                      // rows per pass
  static constexpr int PASSES = (DK + RPP - 1) / RPP;
  static constexpr uint32_t kRed = 2 * RPP * DV * 4;                  // partial S^T k, S^T q
  static constexpr uint32_t kSmem = kStepStages * kStage + kRed + (2 * DK + DV + 8) * 4 + 64 + 128;
};

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kStepThreads, 1) delta_step_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const float *__restrict__ g, const float *__restrict__ beta, float *__restrict__ S,
    T *__restrict__ out, int BH) {
  using Lay = StepLayout<DK, DV, T>;
  constexpr int NT = kStepThreads, TPR = Lay::TPR, RPP = Lay::RPP, PASSES = Lay::PASSES;
  static_assert(Lay::kS % 16 == 0 && Lay::kQ % 16 == 0 && Lay::kV % 16 == 0,
                "bulk copies move multiples of 16 bytes");
  static_assert(DK <= NT && 2 * DV <= NT, "one thread per k, and per column of either sum");

  extern __shared__ uint8_t dsm_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsm_raw) + 127) &
                                            ~static_cast<uintptr_t>(127));
  float *s_red = reinterpret_cast<float *>(sm + kStepStages * Lay::kStage);
  float *s_k = s_red + 2 * RPP * DV;
  float *s_q = s_k + DK;
  float *s_u = s_q + DK;
  float *s_kq = s_u + DV;                       // NT/32 partials of k . q
  uint8_t *bars = reinterpret_cast<uint8_t *>(s_kq + 8);
  const uint32_t bar0 = smem_u32(bars);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 32);

  const int tid = threadIdx.x;
  const int nmine = (BH - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
                    static_cast<int>(gridDim.x);
  auto issue = [&](int i) {
    const long p = blockIdx.x + static_cast<long>(i) * gridDim.x;
    const int st = i % kStepStages;
    const uint32_t base = smem_u32(sm + st * Lay::kStage);
    const uint32_t bar = bar0 + 8 * st;
    mbar_arrive_expect_tx(bar, Lay::kBytes);
    bulk_load(base, S + p * DK * DV, Lay::kS, bar);
    bulk_load(base + Lay::kS, q + p * DK, Lay::kQ, bar);
    bulk_load(base + Lay::kS + Lay::kQ, k + p * DK, Lay::kQ, bar);
    bulk_load(base + Lay::kS + 2 * Lay::kQ, v + p * DV, Lay::kV, bar);
  };
  if (tid == 0) {
    for (int st = 0; st < kStepStages; ++st) mbar_init(bar0 + 8 * st, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < nmine && i < kStepStages; ++i) issue(i);
  }
  __syncthreads();

  const int c4 = tid % TPR;
  const int r0 = tid / TPR;
  int i = 0;
  for (; i < nmine; ++i) {
    const long p = blockIdx.x + static_cast<long>(i) * gridDim.x;
    const int st = i % kStepStages;
    const uint8_t *stage = sm + st * Lay::kStage;
    const float *sS = reinterpret_cast<const float *>(stage);
    const T *sq = reinterpret_cast<const T *>(stage + Lay::kS);
    const T *sk = reinterpret_cast<const T *>(stage + Lay::kS + Lay::kQ);
    const T *sv = reinterpret_cast<const T *>(stage + Lay::kS + 2 * Lay::kQ);
    const float gate = g ? g[p] : 0.f, b = beta[p];

    if (!mbar_wait(bar0 + 8 * st, (i / kStepStages) & 1)) *abort_flag = 1;
    __syncthreads();
    if (*abort_flag) break;
    float kq = 0.f;
    if (tid < DK) {
      const float fk = to_f32(sk[tid]), fq = to_f32(sq[tid]);
      s_k[tid] = fk;
      s_q[tid] = fq;
      kq = fk * fq;
    }
    kq = warp_sum(kq);
    if ((tid & 31) == 0) s_kq[tid >> 5] = kq;
    const float vv = tid < DV ? to_f32(sv[tid]) : 0.f;
    __syncthreads();

    float4 x[PASSES];
    float4 ak = make_float4(0.f, 0.f, 0.f, 0.f), aq = ak;
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
      const int r = r0 + j * RPP;
      if (r < DK) {
        x[j] = *reinterpret_cast<const float4 *>(sS + r * DV + 4 * c4);
        const float fk = s_k[r], fq = s_q[r];
        ak.x = fmaf(fk, x[j].x, ak.x); aq.x = fmaf(fq, x[j].x, aq.x);
        ak.y = fmaf(fk, x[j].y, ak.y); aq.y = fmaf(fq, x[j].y, aq.y);
        ak.z = fmaf(fk, x[j].z, ak.z); aq.z = fmaf(fq, x[j].z, aq.z);
        ak.w = fmaf(fk, x[j].w, ak.w); aq.w = fmaf(fq, x[j].w, aq.w);
      }
    }
    *reinterpret_cast<float4 *>(&s_red[r0 * DV + 4 * c4]) = ak;
    *reinterpret_cast<float4 *>(&s_red[(RPP + r0) * DV + 4 * c4]) = aq;
    // a rounded to fp32 is off by the same 2^-25 at every token of a slow gate, so S
    // takes a - 1; of an a below a half that would be too coarse, and its rounding
    // does not add up.  Taken here, where the gate has come in: at the top of the
    // loop 256 x 32 heads took 194 us.
    const float less = expm1f(gate);
    const bool near = fabsf(less) < 0.5f;
    float a = 1.f + less;
    if (!near) a = expf(gate);
    __syncthreads();
    // every read of this stage is done: refill it with head i + stages
    if (tid == 0 && i + kStepStages < nmine) {
      fence_proxy_async_smem();
      issue(i + kStepStages);
    }
    if (tid < DV) {
      float sk_ = 0.f, sq_ = 0.f, kqs = 0.f;
#pragma unroll 8
      for (int r = 0; r < RPP; ++r) {
        sk_ += s_red[r * DV + tid];
        sq_ += s_red[(RPP + r) * DV + tid];
      }
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) kqs += s_kq[w];
      const float u = b * fmaf(-a, sk_, vv);
      s_u[tid] = u;
      out[p * DV + tid] = from_f32<T>(fmaf(kqs, u, a * sq_));
    }
    __syncthreads();
    const float4 u = *reinterpret_cast<const float4 *>(s_u + 4 * c4);
    float4 *Sp = reinterpret_cast<float4 *>(S + p * DK * DV);
    const auto update = [&](auto decay) {
#pragma unroll
      for (int j = 0; j < PASSES; ++j) {
        const int r = r0 + j * RPP;
        if (r < DK) {
          const float fk = s_k[r];
          __stcs(&Sp[r * TPR + c4],
                 make_float4(fmaf(fk, u.x, decay(x[j].x)), fmaf(fk, u.y, decay(x[j].y)),
                             fmaf(fk, u.z, decay(x[j].z)), fmaf(fk, u.w, decay(x[j].w))));
        }
      }
    };
    if (near) update([&](float s) { return fmaf(less, s, s); });
    else update([&](float s) { return a * s; });
    __syncthreads();
  }
  if (*abort_flag && tid == 0) {
    // drain the copies still in flight (bounded waits)
    for (int j = i; j < nmine && j < i + kStepStages; ++j)
      mbar_wait(bar0 + 8 * (j % kStepStages), (j / kStepStages) & 1);
  }
}

}  // namespace delta
}  // namespace linattn
