// What the host layer's translation units share: argument checks, kernel
// attributes, tensor maps and launch configurations.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>
#include <set>
#include <utility>

#include "../../include/linattn.h"

namespace linattn {
namespace {

using bf16 = __nv_bfloat16;

inline bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

inline size_t elem_size(int dtype) { return dtype == LINATTN_F32 ? 4 : 2; }

// Common checks on the dims struct; returns a status code.
inline int check_dims(const linattn_dims *d, bool use_n) {
  if (!d) return LINATTN_ERR_INVALID;
  if (d->B < 0 || d->H < 0 || (use_n && d->N < 0)) return LINATTN_ERR_INVALID;
  if (d->dtype != LINATTN_BF16 && d->dtype != LINATTN_F32) return LINATTN_ERR_UNSUPPORTED;
  if (d->phi != LINATTN_PHI_ELU1 && d->phi != LINATTN_PHI_IDENTITY) return LINATTN_ERR_UNSUPPORTED;
  if (!supported_dim(d->dk) || !supported_dim(d->dv)) return LINATTN_ERR_UNSUPPORTED;
  const long long n = use_n ? d->N : 1;
  const long long big = static_cast<long long>(d->B) * d->H * n *
                        (d->dk > d->dv ? d->dk : d->dv);
  if (big >= (1ll << 31)) return LINATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(d->B) * d->H * d->dk * d->dv >= (1ll << 31))
    return LINATTN_ERR_UNSUPPORTED;
  return LINATTN_OK;
}

// q and k hold feature vectors already: the kernels apply no feature map
inline bool ident(const linattn_dims *d) { return d->phi == LINATTN_PHI_IDENTITY; }

inline bool bad_eps(float eps) { return !(eps >= 0.f) || !std::isfinite(eps); }

inline int launch_status() {
  return cudaGetLastError() == cudaSuccess ? LINATTN_OK : LINATTN_ERR_CUDA;
}

// Opt a kernel in to more than 48 KB of dynamic shared memory, once per
// (kernel, device).  Keyed by the kernel's address: instantiations that share
// a signature are still distinct kernels.
inline bool set_smem_impl(const void *kernel, int bytes) {
  static std::mutex mu;
  static std::set<std::pair<const void *, int>> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({kernel, dev})) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done.insert({kernel, dev});
  return true;
}

template <typename F>
inline bool set_smem(F *kernel, int bytes) {
  return set_smem_impl(reinterpret_cast<const void *>(kernel), bytes);
}

// ------------------------------------------------------------ tensor maps
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  });
  return fn;
}

// [planes, rows, inner] bf16 tensor; boxes of 64 x box_rows x 1 with 128-byte
// swizzle (64 bf16 = 128 bytes per box row).
inline bool make_map_bf16(CUtensorMap *m, const void *ptr, int inner, int rows, int planes,
                   unsigned box_rows = 128) {
  EncodeTiled enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2,
                                 static_cast<cuuint64_t>(inner) * rows * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Launch configuration with programmatic stream serialization: the grid may
// begin before the previous grid of the stream has finished, and orders
// itself after it with griddepcontrol.wait where it reads that grid's output.
struct ProgrammaticLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  ProgrammaticLaunch(int grid, int block, size_t smem, cudaStream_t s) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

// One buffer of a call: where it lies and how long it is.
struct Span {
  const void *p;
  size_t n;
};

// Every pointer 16-byte aligned; no output over an input or another output.
template <int NI, int NO>
inline bool bad_spans(const Span (&in)[NI], const Span (&out)[NO]) {
  for (const Span &a : in)
    if (!aligned16(a.p)) return true;
  for (int o = 0; o < NO; ++o) {
    if (!aligned16(out[o].p)) return true;
    for (const Span &a : in)
      if (overlaps(out[o].p, out[o].n, a.p, a.n)) return true;
    for (int o2 = o + 1; o2 < NO; ++o2)
      if (overlaps(out[o].p, out[o].n, out[o2].p, out[o2].n)) return true;
  }
  return false;
}

}  // namespace

// linattn.cu: the kernel family chosen for an operation (linattn_set_kernel_choice).
int kernel_choice(int op);

// delta.cu: reads (and with `clear` resets) the error word of its kernels on
// the current device; false when CUDA reports an error.
bool delta_status(bool clear, unsigned int *word);

}  // namespace linattn
