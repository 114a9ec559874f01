// Layer norm and RMS norm of the rows of [rows, d], and their gradients.
//
//   m = mean(x) (layer norm) or 0 (RMS norm),  s = mean((x - m)^2),
//   xh = (x - m) / sqrt(s + eps),  y = w o xh + b
//   dx = (w o dy - [mean(w o dy)] - xh mean(w o dy o xh)) / sqrt(s + eps)
//   dw = sum over rows of dy o xh,  db = sum over rows of dy
// (the bracketed mean for layer norm only).  The backward forms m and s from x
// again: it has the row in registers anyway, and so nothing of the forward has
// to be kept.  The variance is summed from x - m, not as E[x^2] - m^2.
//
// Bound by HBM: a row is read once and written once, everything between stays
// in registers.  TPR threads (a power of two) hold a row, 8 elements each: one
// 16-byte load a thread in bf16, two in fp32, when rows start on 16-byte
// boundaries (VEC); elements TPR apart otherwise, so that a warp still reads
// consecutive ones.  A thread works on `ROWS` rows at a time: their loads are
// in flight together, and with TPR > 32 they share the block barriers of the
// reductions.
//
// dw and db: a thread meets the same columns in every row it takes, so it adds
// them up in registers over a grid-stride loop; a block joins its row groups
// in shared memory and writes one partial row of each, and norm_bwd_sum_kernel
// adds the partial rows in a fixed order (no atomics: the sums do not change
// from run to run).
#pragma once
#include "common.cuh"

namespace linattn {
namespace norm {

constexpr int kMaxD = 8192;
constexpr int kE = 8;                  // elements of a row per thread

template <int TPR>
struct Shape {
  static constexpr int NT = TPR > 256 ? TPR : 256;   // threads per block
  static constexpr int GROUPS = NT / TPR;            // rows side by side in a block
  static constexpr int ROWS = TPR > 256 ? 1 : 2;     // rows per thread and step
};

template <int TPR, bool VEC>
__device__ __forceinline__ int col_of(int lane, int e) {
  return VEC ? lane * kE + e : e * TPR + lane;
}

template <int TPR, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T *row, int lane, int d, bool live,
                                         float (&f)[kE]) {
  if constexpr (VEC) {
#pragma unroll
    for (int e = 0; e < kE; ++e) f[e] = 0.f;
    if (live && lane * kE < d) load8_f32(row + lane * kE, f);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = e * TPR + lane;
      f[e] = live && c < d ? to_f32(row[c]) : 0.f;
    }
  }
}

template <int TPR, bool VEC, typename T>
__device__ __forceinline__ void store_row(T *row, int lane, int d, const float (&f)[kE]) {
  if constexpr (VEC) {
    if (lane * kE < d) {
      if constexpr (sizeof(T) == 2) {
        uint4 w;
        __nv_bfloat162 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w = *reinterpret_cast<uint4 *>(p);
        *reinterpret_cast<uint4 *>(row + lane * kE) = w;
      } else {
        reinterpret_cast<float4 *>(row + lane * kE)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(row + lane * kE)[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int c = e * TPR + lane;
      if (c < d) row[c] = from_f32<T>(f[e]);
    }
  }
}

// Sums of NV values over the TPR threads of each row; every thread gets them.
// With TPR > 32 all threads of the block take part (red: two halves of
// NT / 32 x 2 ROWS floats, `turn` alternates them, so one barrier a call is
// enough: a half is written again two calls later, behind the next barrier).
template <int TPR, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float *red, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (TPR > 32) {
    constexpr int NW = Shape<TPR>::NT / 32, WPR = TPR / 32;
    const int warp = threadIdx.x >> 5;
    float *r = red + turn * NW * 2 * Shape<TPR>::ROWS;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < NV; ++i) r[warp * NV + i] = v[i];
    __syncthreads();
    const int w0 = warp / WPR * WPR;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s += r[(w0 + w) * NV + i];
      v[i] = s;
    }
  }
}

template <int TPR>
constexpr int red_floats() {
  return TPR > 32 ? 2 * (Shape<TPR>::NT / 32) * 2 * Shape<TPR>::ROWS : 1;
}

// x becomes xh (0 in columns past d); returns 1 / sqrt(s + eps) of each row
template <int TPR, bool VEC, int ROWS>
__device__ __forceinline__ void normalise(float (&x)[ROWS][kE], float (&rstd)[ROWS], int lane,
                                          int d, float inv_d, float eps, bool rms, float *red,
                                          int &turn) {
  if (!rms) {
    float s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) s[r] += x[r][e];
    }
    row_sums<TPR, ROWS>(s, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int e = 0; e < kE; ++e)
        x[r][e] = col_of<TPR, VEC>(lane, e) < d ? x[r][e] - s[r] * inv_d : 0.f;
  }
  float s[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    s[r] = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) s[r] = fmaf(x[r][e], x[r][e], s[r]);
  }
  row_sums<TPR, ROWS>(s, red, turn);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    rstd[r] = 1.f / sqrtf(fmaf(s[r], inv_d, eps));
#pragma unroll
    for (int e = 0; e < kE; ++e) x[r][e] *= rstd[r];
  }
}

template <int TPR, bool VEC, typename T>
__global__ void __launch_bounds__(Shape<TPR>::NT) norm_fwd_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
    T *__restrict__ out, long rows, int d, float inv_d, float eps, bool rms) {
  constexpr int ROWS = Shape<TPR>::ROWS, GROUPS = Shape<TPR>::GROUPS;
  __shared__ float red[red_floats<TPR>()];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  int turn = 0;
  float fw[kE], fb[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = col_of<TPR, VEC>(lane, e);
    fw[e] = w && c < d ? w[c] : 1.f;
    fb[e] = b && c < d ? b[c] : 0.f;
  }
  const long step = static_cast<long>(gridDim.x) * GROUPS * ROWS;
  for (long r0 = static_cast<long>(blockIdx.x) * GROUPS * ROWS; r0 < rows; r0 += step) {
    float f[ROWS][kE], rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      load_row<TPR, VEC>(x + row * d, lane, d, row < rows, f[r]);
    }
    normalise<TPR, VEC, ROWS>(f, rstd, lane, d, inv_d, eps, rms, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      if (row >= rows) continue;
#pragma unroll
      for (int e = 0; e < kE; ++e) f[r][e] = fmaf(f[r][e], fw[e], fb[e]);
      store_row<TPR, VEC>(out + row * d, lane, d, f[r]);
    }
  }
}

// part: [blocks][2][d] partial rows of dw and db (NULL when neither is wanted)
template <int TPR, bool VEC, typename T>
__global__ void __launch_bounds__(Shape<TPR>::NT) norm_bwd_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const T *__restrict__ dy,
    T *__restrict__ dx, float *__restrict__ part, long rows, int d, float inv_d, float eps,
    bool rms) {
  constexpr int ROWS = Shape<TPR>::ROWS, GROUPS = Shape<TPR>::GROUPS;
  __shared__ float red[red_floats<TPR>()];
  __shared__ float join[GROUPS > 1 ? Shape<TPR>::NT * kE : 1];
  const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  int turn = 0;
  float fw[kE], aw[kE], ab[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = col_of<TPR, VEC>(lane, e);
    fw[e] = w && c < d ? w[c] : 1.f;
    aw[e] = ab[e] = 0.f;
  }
  const long step = static_cast<long>(gridDim.x) * GROUPS * ROWS;
  for (long r0 = static_cast<long>(blockIdx.x) * GROUPS * ROWS; r0 < rows; r0 += step) {
    float f[ROWS][kE], gy[ROWS][kE], rstd[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      load_row<TPR, VEC>(x + row * d, lane, d, row < rows, f[r]);
      load_row<TPR, VEC>(dy + row * d, lane, d, row < rows, gy[r]);
    }
    normalise<TPR, VEC, ROWS>(f, rstd, lane, d, inv_d, eps, rms, red, turn);
    float s[2 * ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      s[2 * r] = s[2 * r + 1] = 0.f;
      if (r0 + r * GROUPS + grp >= rows) continue;   // no row: f may be 0 / 0
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        aw[e] = fmaf(gy[r][e], f[r][e], aw[e]);
        ab[e] += gy[r][e];
        gy[r][e] *= fw[e];
        s[2 * r] = fmaf(gy[r][e], f[r][e], s[2 * r]);
        s[2 * r + 1] += gy[r][e];
      }
    }
    row_sums<TPR, 2 * ROWS>(s, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      if (row >= rows) continue;
      const float m1 = s[2 * r] * inv_d, m0 = rms ? 0.f : s[2 * r + 1] * inv_d;
#pragma unroll
      for (int e = 0; e < kE; ++e) f[r][e] = rstd[r] * (gy[r][e] - m0 - f[r][e] * m1);
      store_row<TPR, VEC>(dx + row * d, lane, d, f[r]);
    }
  }
  if (!part) return;
  float *pw = part + static_cast<long>(blockIdx.x) * 2 * d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float (&acc)[kE] = which ? ab : aw;
    if constexpr (GROUPS > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kE; ++e) join[e * Shape<TPR>::NT + threadIdx.x] = acc[e];
      __syncthreads();
      if (grp == 0) {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          float s = 0.f;
          for (int o = 0; o < GROUPS; ++o) s += join[e * Shape<TPR>::NT + o * TPR + lane];
          acc[e] = s;
        }
      }
    }
    if (grp == 0)
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int c = col_of<TPR, VEC>(lane, e);
        if (c < d) pw[static_cast<long>(which) * d + c] = acc[e];
      }
  }
}

// dw and db from the blocks' partial rows: 32 columns a block, 32 threads to a
// column, each adding every 32nd partial row
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float *__restrict__ part,
                                                             float *__restrict__ dw,
                                                             float *__restrict__ db, int blocks,
                                                             int d) {
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float *dst = blockIdx.y ? db : dw;
  if (!dst) return;
  float s = 0.f;
  if (c < d)
    for (int i = ty; i < blocks; i += 32)
      s += part[(static_cast<long>(i) * 2 + blockIdx.y) * d + c];
  red[ty][tx] = s;
  __syncthreads();
  s = warp_sum(red[tx][ty]);
  if (tx == 0 && blockIdx.x * 32 + ty < d) dst[blockIdx.x * 32 + ty] = s;
}

}  // namespace norm
}  // namespace linattn
