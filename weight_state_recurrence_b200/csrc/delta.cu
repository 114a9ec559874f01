// The host layer (argument checks, kernel choice, launches) of the gated delta rule.  See
// include/linattn.h for the contract of every entry point.
#include <algorithm>
#include <cstdint>

#include "../../include/linattn.h"
#include "host.cuh"
#include "common.cuh"
#include "sm100.cuh"
#include "delta_simt.cuh"
#include "delta_step.cuh"
#include "delta_tc.cuh"
#include "delta_bwd_tc.cuh"

using namespace linattn;

namespace {

// The checks the delta calls share.  The rule is defined on the vectors as
// they are: dims.phi has to say so.
int check_delta(const linattn_dims *d, bool use_n) {
  const int rc = check_dims(d, use_n);
  if (rc != LINATTN_OK) return rc;
  return d->phi == LINATTN_PHI_IDENTITY ? LINATTN_OK : LINATTN_ERR_UNSUPPORTED;
}

// dst = src, or zeros without a src: the state after no token at all
int copy_state(float *dst, const float *src, size_t bytes, cudaStream_t s) {
  if (!dst) return LINATTN_OK;
  const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                            : cudaMemsetAsync(dst, 0, bytes, s);
  return e == cudaSuccess ? LINATTN_OK : LINATTN_ERR_CUDA;
}

// Blocks of the CUDA-core recurrences have four warps at most, one for each
// scheduler of an SM.  While all of them find an SM of their own, four lanes
// work on a column of S, 32 columns a block; with more heads two lanes, 64
// columns.
bool simt_four_lanes(long heads, int dv) { return heads * (dv < 32 ? 1 : dv / 32) <= num_sms(); }

template <int DK, int L, typename T>
int launch_delta_fwd_simt(const linattn_dims *d, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, const float *S_init, void *out,
                          float *S_final, cudaStream_t s) {
  const int cols = std::min(d->dv, delta::kSimtThreads / L), bytes = sizeof(delta::SimtTile<DK, T>);
  auto *kern = delta::delta_fwd_simt_kernel<DK, L, T>;
  if (!set_smem(kern, bytes)) return LINATTN_ERR_CUDA;
  kern<<<dim3(d->B * d->H, d->dv / cols), cols * L, bytes, s>>>(
      static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v), g, beta,
      S_init, static_cast<T *>(out), S_final, d->N, d->dv);
  return launch_status();
}

template <int DK, typename T>
int launch_delta_fwd_simt(const linattn_dims *d, const void *q, const void *k, const void *v,
                          const float *g, const float *beta, const float *S_init, void *out,
                          float *S_final, cudaStream_t s) {
  auto *launch = simt_four_lanes(static_cast<long>(d->B) * d->H, d->dv)
                     ? launch_delta_fwd_simt<DK, 4, T>
                     : launch_delta_fwd_simt<DK, 2, T>;
  return launch(d, q, k, v, g, beta, S_init, out, S_final, s);
}

template <typename T>
int delta_fwd_simt(const linattn_dims *d, const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const float *S_init, void *out,
                   float *S_final, cudaStream_t s) {
  switch (d->dk) {
    case 16: return launch_delta_fwd_simt<16, T>(d, q, k, v, g, beta, S_init, out, S_final, s);
    case 32: return launch_delta_fwd_simt<32, T>(d, q, k, v, g, beta, S_init, out, S_final, s);
    case 64: return launch_delta_fwd_simt<64, T>(d, q, k, v, g, beta, S_init, out, S_final, s);
    case 128: return launch_delta_fwd_simt<128, T>(d, q, k, v, g, beta, S_init, out, S_final, s);
  }
  return LINATTN_ERR_UNSUPPORTED;
}

// The arguments of one backward call.
struct DeltaBwd {
  const void *q, *k, *v, *dout;
  const float *g, *beta, *S_init, *dS_final;
  void *dq, *dk, *dv;
  float *dg, *dbeta, *dS_init;
};

// Workspace of the CUDA-core backward: the states before and the gradients
// after every chunk, r and du of every token, and what segments of the sequence
// pass on.  Segments need a block each for 32 columns of B, E and M, which must
// find an SM each; they pay when two walks of a segment (4.2 us a chunk of 32
// tokens) and the joining (15 us, 2 a segment) take less than one walk of the
// sequence (8 heads x 1001 tokens, 64 x 32, 6 segments: the call 99 us, in one
// piece 161; 4 x 4096, d = 32: 116 and 459).  The times are those of d = 64; of 432
// calls with sizes of 16 to 128, 1 to 24 heads and 256 to 2048 tokens none was slower
// than in one piece.
struct DeltaSimtWs {
  size_t nch, states, rows, ends, trans, bytes;
  int segs = 1, len;
  explicit DeltaSimtWs(const linattn_dims *d) {
    const size_t BH = static_cast<size_t>(d->B) * d->H;
    nch = (static_cast<size_t>(d->N) + delta::kSimtChunk - 1) / delta::kSimtChunk;
    states = BH * nch * d->dk * d->dv;
    rows = BH * d->N * d->dv;
    len = static_cast<int>(nch);
    const long cols = std::min(d->dv, 32), nb = d->dv / cols, mb = (d->dk + cols - 1) / cols;
    double best = 4.2 * nch;
    const long sms = num_sms();
    for (int g = 3; g <= 64 && static_cast<long>(BH) * (2 * (g - 1) * nb + (g - 2) * mb) <= sms; ++g) {
      const int l = static_cast<int>((nch + g - 1) / g);
      if (static_cast<size_t>(g - 1) * l >= nch) continue;   // no empty segments
      const double t = 8.4 * l + 15. + 2. * g;
      if (t < best) {
        best = t;
        segs = g;
        len = l;
      }
    }
    ends = segs > 1 ? (segs - 1) * BH * d->dk * d->dv : 0;
    trans = segs > 1 ? (segs - 2) * BH * d->dk * d->dk : 0;
    bytes = (2 * (states + rows + ends) + trans) * sizeof(float);
  }
};

template <int DK, int DV, typename T>
int launch_delta_grad_simt(const linattn_dims *d, const DeltaBwd &a, const float *keep_S,
                           const float *keep_D, const float *keep_r, const float *keep_du, int nch,
                           cudaStream_t s) {
  auto *kern = delta::delta_bwd_grad_simt_kernel<DK, DV, T>;
  const int bytes = delta::delta_grad_simt_smem_floats<DK, DV>() * 4;
  if (!set_smem(kern, bytes)) return LINATTN_ERR_CUDA;
  kern<<<d->B * d->H * nch, delta::kSimtGradThreads, bytes, s>>>(
      static_cast<const T *>(a.q), static_cast<const T *>(a.k), static_cast<const T *>(a.dout), a.g,
      a.beta, keep_S, keep_D, keep_r, keep_du, static_cast<T *>(a.dq), static_cast<T *>(a.dk), a.dg,
      a.dbeta, d->N, nch);
  return launch_status();
}

template <int DK, int L, typename T>
int launch_delta_sweep_simt(const linattn_dims *d, const DeltaBwd &a, const DeltaSimtWs &w, float *ws,
                            cudaStream_t s) {
  const int BH = d->B * d->H, cols = std::min(d->dv, delta::kSimtThreads / L);
  const int bytes = sizeof(delta::SimtTile<DK, T>);
  float *keep_S = ws, *keep_D = ws + w.states;
  float *keep_r = keep_D + w.states, *keep_du = keep_r + w.rows;
  float *ends = keep_du + w.rows;
  const delta::SimtSegments x{ends, ends + w.ends, ends + 2 * w.ends, w.segs, w.len};
  const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k);
  const T *v = static_cast<const T *>(a.v), *dout = static_cast<const T *>(a.dout);
  auto *sweep = delta::delta_sweep_simt_kernel<DK, L, T, false>;
  if constexpr (L == 4) {
    if (w.segs > 1) {
      sweep = delta::delta_sweep_simt_kernel<DK, L, T, true>;
      auto *trans = delta::delta_transition_simt_kernel<DK, L, T>;
      if (!set_smem(trans, bytes)) return LINATTN_ERR_CUDA;
      const int parts = 2 * (w.segs - 1) + w.segs - 2, most = std::max(d->dv, DK);
      trans<<<dim3(BH * parts, (most + cols - 1) / cols), cols * L, bytes, s>>>(
          q, k, v, dout, a.g, a.beta, a.S_init, a.dS_final, x, BH, d->N, d->dv);
      if (cudaGetLastError() != cudaSuccess) return LINATTN_ERR_CUDA;
      auto *join = delta::delta_join_simt_kernel<DK>;
      if (!set_smem(join, delta::simt_join_smem<DK>())) return LINATTN_ERR_CUDA;
      join<<<dim3(BH, d->dv / 16, 2), 256, delta::simt_join_smem<DK>(), s>>>(x, BH, d->dv);
      if (cudaGetLastError() != cudaSuccess) return LINATTN_ERR_CUDA;
    }
  }
  if (!set_smem(sweep, bytes)) return LINATTN_ERR_CUDA;
  sweep<<<dim3(2 * BH * w.segs, d->dv / cols), cols * L, bytes, s>>>(
      q, k, v, dout, a.g, a.beta, a.S_init, a.dS_final, static_cast<T *>(a.dv), a.dS_init, keep_S,
      keep_D, keep_r, keep_du, x, BH, d->N, d->dv);
  return launch_status();
}

template <int DK, typename T>
int launch_delta_bwd_simt(const linattn_dims *d, const DeltaBwd &a, float *ws, cudaStream_t s) {
  const DeltaSimtWs w(d);
  float *keep_S = ws, *keep_D = ws + w.states;
  float *keep_r = keep_D + w.states, *keep_du = keep_r + w.rows;
  const bool four = w.segs > 1 || simt_four_lanes(2L * d->B * d->H, d->dv);
  const int rc =
      (four ? launch_delta_sweep_simt<DK, 4, T> : launch_delta_sweep_simt<DK, 2, T>)(d, a, w, ws, s);
  if (rc != LINATTN_OK) return rc;
  const int nch = static_cast<int>(w.nch);
  switch (d->dv) {
    case 16: return launch_delta_grad_simt<DK, 16, T>(d, a, keep_S, keep_D, keep_r, keep_du, nch, s);
    case 32: return launch_delta_grad_simt<DK, 32, T>(d, a, keep_S, keep_D, keep_r, keep_du, nch, s);
    case 64: return launch_delta_grad_simt<DK, 64, T>(d, a, keep_S, keep_D, keep_r, keep_du, nch, s);
    case 128: return launch_delta_grad_simt<DK, 128, T>(d, a, keep_S, keep_D, keep_r, keep_du, nch, s);
  }
  return LINATTN_ERR_UNSUPPORTED;
}

template <typename T>
int delta_bwd_simt(const linattn_dims *d, const DeltaBwd &a, float *ws, cudaStream_t s) {
  switch (d->dk) {
    case 16: return launch_delta_bwd_simt<16, T>(d, a, ws, s);
    case 32: return launch_delta_bwd_simt<32, T>(d, a, ws, s);
    case 64: return launch_delta_bwd_simt<64, T>(d, a, ws, s);
    case 128: return launch_delta_bwd_simt<128, T>(d, a, ws, s);
  }
  return LINATTN_ERR_UNSUPPORTED;
}

template <int DK, int DV, typename T>
int launch_delta_step(const linattn_dims *d, const void *q, const void *k, const void *v,
                      const float *g, const float *beta, float *S, void *out, cudaStream_t s) {
  auto *kern = delta::delta_step_kernel<DK, DV, T>;
  const int bytes = static_cast<int>(delta::StepLayout<DK, DV, T>::kSmem);
  if (!set_smem(kern, bytes)) return LINATTN_ERR_CUDA;
  const int BH = d->B * d->H, sms = num_sms();
  if (sms <= 0) return LINATTN_ERR_CUDA;
  kern<<<BH < sms ? BH : sms, delta::kStepThreads, bytes, s>>>(
      static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v), g, beta, S,
      static_cast<T *>(out), BH);
  return launch_status();
}

template <int DK, typename T>
int delta_step_dv(const linattn_dims *d, const void *q, const void *k, const void *v,
                  const float *g, const float *beta, float *S, void *out, cudaStream_t s) {
  switch (d->dv) {
    case 16: return launch_delta_step<DK, 16, T>(d, q, k, v, g, beta, S, out, s);
    case 32: return launch_delta_step<DK, 32, T>(d, q, k, v, g, beta, S, out, s);
    case 64: return launch_delta_step<DK, 64, T>(d, q, k, v, g, beta, S, out, s);
    case 128: return launch_delta_step<DK, 128, T>(d, q, k, v, g, beta, S, out, s);
  }
  return LINATTN_ERR_UNSUPPORTED;
}

template <typename T>
int delta_step_dispatch(const linattn_dims *d, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, float *S, void *out, cudaStream_t s) {
  switch (d->dk) {
    case 16: return delta_step_dv<16, T>(d, q, k, v, g, beta, S, out, s);
    case 32: return delta_step_dv<32, T>(d, q, k, v, g, beta, S, out, s);
    case 64: return delta_step_dv<64, T>(d, q, k, v, g, beta, S, out, s);
    case 128: return delta_step_dv<128, T>(d, q, k, v, g, beta, S, out, s);
  }
  return LINATTN_ERR_UNSUPPORTED;
}

}  // namespace

namespace {

// A launch that may begin while the kernel before it on the stream ends: every
// kernel launched so waits for that one (grid_dependency_wait) before it reads
// what others wrote.
template <typename... P, typename... A>
bool launch_after(void (*kern)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, A... args) {
  ProgrammaticLaunch pl(1, block, smem, s);
  pl.cfg.gridDim = grid;
  return cudaLaunchKernelEx(&pl.cfg, kern, P(args)...) == cudaSuccess;
}

// bf16 with d_k and d_v in {64, 128} takes the tensor-core kernels.
bool use_tc_delta(const linattn_dims *d) {
  if (kernel_choice(LINATTN_OP_DELTA) == LINATTN_KERNEL_CUDA_CORES) return false;
  return d->dtype == LINATTN_BF16 && (d->dk == 64 || d->dk == 128) && (d->dv == 64 || d->dv == 128);
}

size_t delta_chunks(const linattn_dims *d) {
  return (static_cast<size_t>(d->N) + delta::C - 1) / delta::C;
}

// one record per chunk and head (delta_tc.cuh)
size_t delta_rec_bytes(const linattn_dims *d) {
  return static_cast<size_t>(d->B) * d->H * delta_chunks(d) * delta::kRecord;
}

// How the forward cuts the chunks of a sequence, by what its parts were
// measured to take at d = 128: a chunk 3.4 us of chain, 0.85 of that without
// outputs, and 0.0183 us of prep per head on the whole device.
//
// Segments (few heads): every segment's own transition first, S -> M S + B, a CTA
// each for B and M; the states between them; then all segments at once with their
// outputs.  It takes 2 segs - 3 and segs CTAs per head, which must not be more
// than there are SMs, and pays when 1.85 / segs of the chain, the joining (2.2 us
// a segment) and 25 us of launches take less than the chain (32 heads x 256
// chunks, d = 128, 3 segments: 613 us, in one piece 902; 16 heads x 64 chunks,
// d = 64, 6 segments: 98, in one piece 197).  The last segment's transition is
// not asked for, so its chunks are prepared beside the others' transitions
// where the SMs left free do that in their time (30 us of the first of these).
//
// Slabs (more heads, SMs left free all the same): while the chain walks the first
// slab, prep works on the second beside it.  The first is as long as prep needs
// for the second, and a tenth; a second launch of the chain costs 10 us, so there
// is one only where it hides more than 25 us of prep (64 heads x 64 chunks: 269 us
// in one piece, 250 in two).
//
// The times are those of d = 128; of 412 calls with d_k and d_v of 64 and 128, 1 to
// 130 heads and 512 to 8192 tokens none was slower than in one piece.
struct DeltaPlan {
  int segs = 1, len = 0, first = 0;   // segments of len chunks; chunks prepared first
  explicit DeltaPlan(const linattn_dims *d) {
    constexpr double kChain = 3.4, kPrep = 0.0183;
    const int BH = d->B * d->H, nch = static_cast<int>(delta_chunks(d)), sms = num_sms();
    len = first = nch;
    if (BH == 0 || BH >= sms || nch < 8) return;
    double best = kChain * nch, hidden = 0;
    const double ratio = kPrep / kChain * BH * sms / (sms - BH);   // prep beside the chain to it
    const int f = std::max(2, static_cast<int>(1.1 * ratio / (1 + ratio) * nch + 0.5));
    if (f < nch && (nch - f) * BH * kPrep > 25.) {
      first = f;
      hidden = (nch - f) * BH * kPrep - 10.;
    }
    best -= hidden;
    for (int g = 3; g <= 64 && BH * (2 * g - 3) <= sms && g <= nch; ++g) {
      const int l = (nch + g - 1) / g;
      if ((nch + l - 1) / l != g) continue;   // no empty segments
      const int spare = sms - BH * (2 * g - 3);
      const double last = (nch - (g - 1) * l) * BH * kPrep;   // prep of the last segment
      const bool beside = last > 10. && last * sms < 0.85 * kChain * l * spare;
      const double t = 1.85 * kChain * l + 2.2 * g + 25. - (beside ? last - 5. : 0.);
      if (t < best) {
        best = t;
        segs = g;
        len = l;
        first = beside ? (g - 1) * l : nch;
      }
    }
  }
  // a state per head between slabs, or the segments' states and transitions
  size_t bytes(const linattn_dims *d) const {
    const size_t BH = static_cast<size_t>(d->B) * d->H, S = BH * d->dk * d->dv * 4;
    if (segs > 1) return (segs - 1) * S + (segs - 2) * BH * d->dk * d->dk * 4;
    return first < len ? S : 0;
  }
};

size_t delta_fwd_bytes(const linattn_dims *d) { return delta_rec_bytes(d) + DeltaPlan(d).bytes(d); }

template <int DKP>
int launch_delta_fwd_tc(const linattn_dims *d, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const float *S_init, void *out,
                        float *S_final, uint8_t *rec, cudaStream_t s) {
  const int BH = d->B * d->H, nch = static_cast<int>(delta_chunks(d));
  CUtensorMap mq, mk, mv, mo;
  if (!make_map_bf16(&mq, q, d->dk, d->N, BH, delta::C) ||
      !make_map_bf16(&mo, out, d->dv, d->N, BH, delta::C) ||
      !make_map_bf16(&mk, k, d->dk, d->N, BH, delta::C) ||
      !make_map_bf16(&mv, v, d->dv, d->N, BH, delta::C))
    return LINATTN_ERR_CUDA;
  auto *prep = delta::prep::delta_prep_kernel<DKP>;
  auto *chain = delta::chain::delta_chain_kernel<DKP, false>;
  auto *only = delta::chain::delta_chain_kernel<DKP, true>;
  if (!set_smem(prep, static_cast<int>(delta::prep::kSmemBytes)) ||
      !set_smem(chain, static_cast<int>(delta::chain::kSmemBytes)) ||
      !set_smem(only, static_cast<int>(delta::chain::kSmemBytes)))
    return LINATTN_ERR_CUDA;
  const DeltaPlan plan(d);
  float *state = reinterpret_cast<float *>(rec + delta_rec_bytes(d));
  const int rest = nch - plan.first;
  prep<<<BH * plan.first, delta::prep::NT, delta::prep::kSmemBytes, s>>>(mq, mk, g, beta, rec, d->N,
                                                                         nch, 0, plan.first, 0);
  if (cudaGetLastError() != cudaSuccess) return LINATTN_ERR_CUDA;
  auto prep_rest = [&] {   // beside the grid launched before it
    return launch_after(prep, BH * rest, delta::prep::NT, delta::prep::kSmemBytes, s, mq, mk, g,
                        beta, rec, d->N, nch, plan.first, rest, 1);
  };
  delta::chain::Args a{rec, S_init, state, nullptr, S_final, nch, 0, plan.first, 1, BH, d->dv};
  if (plan.segs > 1) {
    a.len = plan.len;
    a.segs = plan.segs;
    a.trans = state + static_cast<size_t>(plan.segs - 1) * BH * d->dk * d->dv;
    if (!launch_after(only, BH * (2 * plan.segs - 3), delta::chain::NT, delta::chain::kSmemBytes, s,
                      mq, mk, mv, mo, a) ||
        (rest && !prep_rest()) ||
        !launch_after(delta::chain::delta_carry_kernel<64 * DKP>, dim3(BH, d->dv / 16),
                      2 * delta::chain::kCarryParts * 64 * DKP, 0, s, a.carry, a.trans, a.segs, BH,
                      d->dv))
      return LINATTN_ERR_CUDA;
    return launch_after(chain, BH * plan.segs, delta::chain::NT, delta::chain::kSmemBytes, s, mq,
                        mk, mv, mo, a)
               ? LINATTN_OK
               : LINATTN_ERR_CUDA;
  }
  if (rest) a.S_final = state;
  if (!launch_after(chain, BH, delta::chain::NT, delta::chain::kSmemBytes, s, mq, mk, mv, mo, a))
    return LINATTN_ERR_CUDA;
  if (rest) {
    if (!prep_rest()) return LINATTN_ERR_CUDA;
    a.S_init = state;
    a.S_final = S_final;
    a.c0 = plan.first;
    a.len = rest;
    chain<<<BH, delta::chain::NT, delta::chain::kSmemBytes, s>>>(mq, mk, mv, mo, a);
    if (cudaGetLastError() != cudaSuccess) return LINATTN_ERR_CUDA;
  }
  return LINATTN_OK;
}

}  // namespace

extern "C" size_t linattn_delta_fwd_workspace(const linattn_dims *d) {
  if (check_delta(d, true) != LINATTN_OK || !use_tc_delta(d)) return 0;
  if (static_cast<size_t>(d->B) * d->H * d->N == 0) return 0;
  return delta_fwd_bytes(d);
}

extern "C" int linattn_delta_fwd(const linattn_dims *d, const void *q, const void *k,
                                 const void *v, const float *g, const float *beta,
                                 const float *S_init, void *out, float *S_final,
                                 void *workspace, size_t workspace_bytes,
                                 linattn_stream_t stream) {
  const int rc = check_delta(d, true);
  if (rc != LINATTN_OK) return rc;
  const size_t BH = static_cast<size_t>(d->B) * d->H;
  if (BH == 0) return LINATTN_OK;
  const size_t es = elem_size(d->dtype), tok = BH * d->N;
  const size_t nk = tok * d->dk * es, nv = tok * d->dv * es, nS = BH * d->dk * d->dv * 4;
  if (d->N > 0 && (!q || !k || !v || !beta || !out)) return LINATTN_ERR_INVALID;
  const size_t need = linattn_delta_fwd_workspace(d);
  if (need && (!workspace || workspace_bytes < need)) return LINATTN_ERR_INVALID;
  const Span in[] = {{q, nk}, {k, nk}, {v, nv}, {g, tok * 4}, {beta, tok * 4}, {S_init, nS}};
  const Span outs[] = {{out, nv}, {S_final, nS}, {workspace, workspace ? workspace_bytes : 0}};
  if (bad_spans(in, outs)) return LINATTN_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->N == 0) return copy_state(S_final, S_init, nS, s);
  if (use_tc_delta(d)) {
    auto *launch = d->dk == 128 ? launch_delta_fwd_tc<2> : launch_delta_fwd_tc<1>;
    return launch(d, q, k, v, g, beta, S_init, out, S_final, static_cast<uint8_t *>(workspace), s);
  }
  if (d->dtype == LINATTN_F32)
    return delta_fwd_simt<float>(d, q, k, v, g, beta, S_init, out, S_final, s);
  return delta_fwd_simt<bf16>(d, q, k, v, g, beta, S_init, out, S_final, s);
}

namespace {

// Workspace of the tensor-core backward: the chunks' records, the states and
// their gradients at every chunk, r and du of every token, the last three as
// a hi and a lo array of bf16 each.  The arrays start on 32 bytes (the sweeps'
// stores of 32), wherever in its first 16 bytes the workspace does.
struct DeltaTcWs {
  size_t rec, states, rows, bytes;
  explicit DeltaTcWs(const linattn_dims *d) {
    const size_t BH = static_cast<size_t>(d->B) * d->H;
    rec = delta_rec_bytes(d);
    states = BH * delta_chunks(d) * d->dk * d->dv;
    rows = BH * d->N * d->dv;
    bytes = rec + (4 * states + 4 * rows) * sizeof(bf16) + 16;
  }
};

template <int DKP>
int launch_delta_bwd_tc(const linattn_dims *d, const DeltaBwd &a, uint8_t *ws, cudaStream_t s) {
  const DeltaTcWs w(d);
  ws += reinterpret_cast<uintptr_t>(ws) & 16u;
  const int BH = d->B * d->H, nch = static_cast<int>(delta_chunks(d)), planes = BH * nch;
  bf16 *p = reinterpret_cast<bf16 *>(ws + w.rec);
  const delta::Kept kept{p, p + w.states, p + 2 * w.states, p + 3 * w.states};
  bf16 *rh = p + 4 * w.states, *rl = rh + w.rows, *uh = rl + w.rows, *ul = uh + w.rows;
  CUtensorMap mq, mk, mv, mo, mdv, mrh, mrl, muh, mul, msh, msl, mdh, mdl, mdq, mdk;
  auto tokens = [&](CUtensorMap *m, const void *x, int inner) {
    return make_map_bf16(m, x, inner, d->N, BH, delta::C);
  };
  auto states = [&](CUtensorMap *m, const void *x) {
    return make_map_bf16(m, x, d->dk, d->dv, planes, 64);
  };
  if (!tokens(&mq, a.q, d->dk) || !tokens(&mk, a.k, d->dk) || !tokens(&mv, a.v, d->dv) ||
      !tokens(&mo, a.dout, d->dv) || !tokens(&mdv, a.dv, d->dv) || !tokens(&mrh, rh, d->dv) ||
      !tokens(&mrl, rl, d->dv) || !tokens(&muh, uh, d->dv) || !tokens(&mul, ul, d->dv) ||
      !states(&msh, kept.s_hi) || !states(&msl, kept.s_lo) || !states(&mdh, kept.d_hi) ||
      !states(&mdl, kept.d_lo) || !tokens(&mdq, a.dq, d->dk) || !tokens(&mdk, a.dk, d->dk))
    return LINATTN_ERR_CUDA;
  auto *prep = delta::prep::delta_prep_kernel<DKP>;
  auto *sweep = delta::sweep::delta_sweep_kernel<DKP>;
  auto *grad = delta::grad::delta_grad_kernel<DKP>;
  if (!set_smem(prep, static_cast<int>(delta::prep::kSmemBytes)) ||
      !set_smem(sweep, static_cast<int>(delta::sweep::kSmemBytes)) ||
      !set_smem(grad, static_cast<int>(delta::grad::kSmemBytes)))
    return LINATTN_ERR_CUDA;
  prep<<<planes, delta::prep::NT, delta::prep::kSmemBytes, s>>>(mq, mk, a.g, a.beta, ws, d->N, nch,
                                                                0, nch, 0);
  if (cudaGetLastError() != cudaSuccess) return LINATTN_ERR_CUDA;
  const delta::grad::Args ga{ws, a.dg, a.dbeta, d->N, nch, d->dv};
  if (!launch_after(sweep, 2 * BH, delta::sweep::NT, delta::sweep::kSmemBytes, s, mq, mk, mv, mo, mrh,
                    mrl, muh, mul, mdv, msh, msl, mdh, mdl, ws, a.S_init, a.dS_final, a.dS_init, kept,
                    BH, nch, d->dv) ||
      !launch_after(grad, planes, delta::grad::NT, delta::grad::kSmemBytes, s, mq, mk, mo, mrh, mrl,
                    muh, mul, msh, msl, mdh, mdl, mdq, mdk, ga))
    return LINATTN_ERR_CUDA;
  return LINATTN_OK;
}

}  // namespace

extern "C" size_t linattn_delta_bwd_workspace(const linattn_dims *d) {
  if (check_delta(d, true) != LINATTN_OK) return 0;
  if (static_cast<size_t>(d->B) * d->H * d->N == 0) return 0;
  return use_tc_delta(d) ? DeltaTcWs(d).bytes : DeltaSimtWs(d).bytes;
}

extern "C" int linattn_delta_bwd(const linattn_dims *d, const void *q, const void *k,
                                 const void *v, const float *g, const float *beta,
                                 const float *S_init, const void *dout, const float *dS_final,
                                 void *dq, void *dk, void *dv, float *dg, float *dbeta,
                                 float *dS_init, void *workspace, size_t workspace_bytes,
                                 linattn_stream_t stream) {
  const int rc = check_delta(d, true);
  if (rc != LINATTN_OK) return rc;
  const size_t BH = static_cast<size_t>(d->B) * d->H;
  if (BH == 0) return LINATTN_OK;
  const size_t es = elem_size(d->dtype), tok = BH * d->N;
  const size_t nk = tok * d->dk * es, nv = tok * d->dv * es, nS = BH * d->dk * d->dv * 4;
  if (d->N > 0 && (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta || !workspace))
    return LINATTN_ERR_INVALID;
  if (workspace_bytes < linattn_delta_bwd_workspace(d)) return LINATTN_ERR_INVALID;
  const Span in[] = {{q, nk},       {k, nk},        {v, nv},       {g, tok * 4},
                     {beta, tok * 4}, {S_init, nS}, {dout, nv},    {dS_final, nS}};
  const Span outs[] = {{dq, nk},        {dk, nk},       {dv, nv}, {dg, tok * 4},
                       {dbeta, tok * 4}, {dS_init, nS},
                       {workspace, workspace ? workspace_bytes : 0}};
  if (bad_spans(in, outs)) return LINATTN_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->N == 0) return copy_state(dS_init, dS_final, nS, s);
  const DeltaBwd a{q, k, v, dout, g, beta, S_init, dS_final, dq, dk, dv, dg, dbeta, dS_init};
  if (use_tc_delta(d)) {
    auto *launch = d->dk == 128 ? launch_delta_bwd_tc<2> : launch_delta_bwd_tc<1>;
    return launch(d, a, static_cast<uint8_t *>(workspace), s);
  }
  if (d->dtype == LINATTN_F32) return delta_bwd_simt<float>(d, a, static_cast<float *>(workspace), s);
  return delta_bwd_simt<bf16>(d, a, static_cast<float *>(workspace), s);
}

extern "C" int linattn_delta_step(const linattn_dims *d, const void *q, const void *k,
                                  const void *v, const float *g, const float *beta, float *S,
                                  void *out, linattn_stream_t stream) {
  const int rc = check_delta(d, false);
  if (rc != LINATTN_OK) return rc;
  const size_t BH = static_cast<size_t>(d->B) * d->H;
  if (BH == 0) return LINATTN_OK;
  if (!q || !k || !v || !beta || !S || !out) return LINATTN_ERR_INVALID;
  const size_t es = elem_size(d->dtype);
  const size_t nk = BH * d->dk * es, nv = BH * d->dv * es, nS = BH * d->dk * d->dv * 4;
  const Span in[] = {{q, nk}, {k, nk}, {v, nv}, {g, BH * 4}, {beta, BH * 4}};
  const Span outs[] = {{out, nv}, {S, nS}};
  if (bad_spans(in, outs)) return LINATTN_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->dtype == LINATTN_F32) return delta_step_dispatch<float>(d, q, k, v, g, beta, S, out, s);
  return delta_step_dispatch<bf16>(d, q, k, v, g, beta, S, out, s);
}

bool linattn::delta_status(bool clear, unsigned int *word) {
  if (cudaMemcpyFromSymbol(word, g_status, sizeof(*word)) != cudaSuccess) return false;
  const unsigned int zero = 0;
  return !clear || cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) == cudaSuccess;
}
