// The host layer (argument checks, kernel choice, launches) of the row norms.  See
// include/linattn.h for the contract of every entry point.
#include <cstdint>

#include "../../include/linattn.h"
#include "host.cuh"
#include "common.cuh"
#include "norm.cuh"

using namespace linattn;

namespace {

// Threads to a row: a power of two with 8 elements each.
int norm_tpr(int d) {
  int t = 1;
  while (t * norm::kE < d) t *= 2;
  return t;
}

// Blocks of a call: as many as share the device, or fewer when there are fewer rows.
long long norm_blocks(long long rows, int rows_per_block, int per_sm) {
  const long long need = (rows + rows_per_block - 1) / rows_per_block;
  const long long most = static_cast<long long>(num_sms()) * per_sm;
  return need < most ? need : most;
}
template <int TPR>
long long norm_blocks_of(long long rows, bool bwd) {
  using S = norm::Shape<TPR>;
  return bwd ? norm_blocks(rows, S::GROUPS * S::BWD_ROWS, S::PER_SM)
             : norm_blocks(rows, S::GROUPS * S::FWD_ROWS, S::FWD_GRID);
}
long long norm_blocks(long long rows, int d, bool bwd) {
  switch (norm_tpr(d)) {
#define LINATTN_NORM_CASE(TPR) \
  case TPR: return norm_blocks_of<TPR>(rows, bwd);
    LINATTN_NORM_CASE(1)
    LINATTN_NORM_CASE(2)
    LINATTN_NORM_CASE(4)
    LINATTN_NORM_CASE(8)
    LINATTN_NORM_CASE(16)
    LINATTN_NORM_CASE(32)
    LINATTN_NORM_CASE(64)
    LINATTN_NORM_CASE(128)
    LINATTN_NORM_CASE(256)
    LINATTN_NORM_CASE(512)
    LINATTN_NORM_CASE(1024)
#undef LINATTN_NORM_CASE
  }
  return 0;
}

bool norm_kind_ok(int kind) { return kind == LINATTN_NORM_LAYER || kind == LINATTN_NORM_RMS; }

int check_norm(long long rows, int d, int kind, int dtype, float eps) {
  if (rows < 0 || d < 1) return LINATTN_ERR_INVALID;
  if (bad_eps(eps)) return LINATTN_ERR_INVALID;
  if (dtype != LINATTN_BF16 && dtype != LINATTN_F32) return LINATTN_ERR_UNSUPPORTED;
  if (!norm_kind_ok(kind) || d > norm::kMaxD) return LINATTN_ERR_UNSUPPORTED;
  if (rows >= (1LL << 40) / d) return LINATTN_ERR_UNSUPPORTED;
  return LINATTN_OK;
}

struct NormArgs {
  const void *x, *dy;
  const float *w, *b;
  void *out;
  float *part;
  long long rows;
  int d, blocks;
  float eps;
  bool rms;
};

template <int TPR, bool VEC, typename T>
int launch_norm(const NormArgs &a, cudaStream_t s) {
  constexpr int NT = norm::Shape<TPR>::NT;
  const float inv_d = 1.f / static_cast<float>(a.d);
  if (a.dy)
    norm::norm_bwd_kernel<TPR, VEC, T><<<a.blocks, NT, 0, s>>>(
        static_cast<const T *>(a.x), a.w, static_cast<const T *>(a.dy), static_cast<T *>(a.out),
        a.part, static_cast<long>(a.rows), a.d, inv_d, a.eps, a.rms);
  else
    norm::norm_fwd_kernel<TPR, VEC, T><<<a.blocks, NT, 0, s>>>(
        static_cast<const T *>(a.x), a.w, a.b, static_cast<T *>(a.out),
        static_cast<long>(a.rows), a.d, inv_d, a.eps, a.rms);
  return launch_status();
}

template <typename T>
int norm_dispatch(const NormArgs &a, cudaStream_t s) {
  const bool vec = a.d * sizeof(T) % 16 == 0 && a.d % norm::kE == 0;
  switch (norm_tpr(a.d)) {
#define LINATTN_NORM_CASE(TPR) \
  case TPR: return vec ? launch_norm<TPR, true, T>(a, s) : launch_norm<TPR, false, T>(a, s);
    LINATTN_NORM_CASE(1)
    LINATTN_NORM_CASE(2)
    LINATTN_NORM_CASE(4)
    LINATTN_NORM_CASE(8)
    LINATTN_NORM_CASE(16)
    LINATTN_NORM_CASE(32)
    LINATTN_NORM_CASE(64)
    LINATTN_NORM_CASE(128)
    LINATTN_NORM_CASE(256)
    LINATTN_NORM_CASE(512)
    LINATTN_NORM_CASE(1024)
#undef LINATTN_NORM_CASE
  }
  return LINATTN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" int linattn_norm_fwd(long long rows, int d, int kind, int dtype, const void *x,
                                const float *weight, const float *bias, float eps, void *out,
                                linattn_stream_t stream) {
  const int rc = check_norm(rows, d, kind, dtype, eps);
  if (rc != LINATTN_OK) return rc;
  if (rows == 0) return LINATTN_OK;
  if (!x || !out) return LINATTN_ERR_INVALID;
  const size_t nx = static_cast<size_t>(rows) * d * elem_size(dtype), nw = static_cast<size_t>(d) * 4;
  const Span in[] = {{x, nx}, {weight, nw}, {bias, nw}};
  const Span outs[] = {{out, nx}};
  if (bad_spans(in, outs)) return LINATTN_ERR_INVALID;
  const long long blocks = norm_blocks(rows, d, false);
  if (blocks <= 0) return LINATTN_ERR_CUDA;
  const NormArgs a{x, nullptr, weight, bias, out, nullptr, rows, d, static_cast<int>(blocks), eps,
                   kind == LINATTN_NORM_RMS};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == LINATTN_F32 ? norm_dispatch<float>(a, s) : norm_dispatch<bf16>(a, s);
}

extern "C" size_t linattn_norm_bwd_workspace(long long rows, int d) {
  if (check_norm(rows, d, LINATTN_NORM_LAYER, LINATTN_F32, 0.f) != LINATTN_OK || rows == 0) return 0;
  const long long blocks = norm_blocks(rows, d, true);
  return blocks <= 0 ? 0 : static_cast<size_t>(blocks) * 2 * d * sizeof(float);
}

extern "C" int linattn_norm_bwd(long long rows, int d, int kind, int dtype, const void *x,
                                const float *weight, float eps, const void *dy, void *dx,
                                float *dweight, float *dbias, void *workspace,
                                size_t workspace_bytes, linattn_stream_t stream) {
  const int rc = check_norm(rows, d, kind, dtype, eps);
  if (rc != LINATTN_OK) return rc;
  const bool sums = dweight || dbias;
  if (rows > 0 && (!x || !dy || !dx)) return LINATTN_ERR_INVALID;
  const size_t nx = static_cast<size_t>(rows) * d * elem_size(dtype), nw = static_cast<size_t>(d) * 4;
  const Span in[] = {{x, nx}, {weight, nw}, {dy, nx}};
  const Span outs[] = {{dx, nx}, {dweight, nw}, {dbias, nw},
                       {workspace, workspace ? workspace_bytes : 0}};
  if (bad_spans(in, outs)) return LINATTN_ERR_INVALID;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if ((dweight && cudaMemsetAsync(dweight, 0, nw, s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, nw, s) != cudaSuccess))
      return LINATTN_ERR_CUDA;
    return LINATTN_OK;
  }
  const long long blocks = norm_blocks(rows, d, true);
  if (sums && (!workspace || workspace_bytes < static_cast<size_t>(blocks) * 2 * d * sizeof(float)))
    return LINATTN_ERR_INVALID;
  if (blocks <= 0) return LINATTN_ERR_CUDA;
  float *part = sums ? static_cast<float *>(workspace) : nullptr;
  const NormArgs a{x, dy, weight, nullptr, dx, part, rows, d, static_cast<int>(blocks), eps,
                   kind == LINATTN_NORM_RMS};
  const int st = dtype == LINATTN_F32 ? norm_dispatch<float>(a, s) : norm_dispatch<bf16>(a, s);
  if (st != LINATTN_OK || !sums) return st;
  ProgrammaticLaunch pl(1, 1024, 0, s);
  pl.cfg.gridDim = dim3((d + 31) / 32, 2);
  if (cudaLaunchKernelEx(&pl.cfg, norm::norm_bwd_sum_kernel, static_cast<const float *>(part),
                         dweight, dbias, static_cast<int>(blocks), d) != cudaSuccess)
    return LINATTN_ERR_CUDA;
  return launch_status();
}
