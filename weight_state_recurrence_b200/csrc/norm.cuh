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
// from run to run).  Above d = 4096 a block has 1024 threads of 64 registers, and the
// backward spills: 76 bytes a thread in fp32, with odd widths 144 and in bf16 200.
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace linattn {
namespace norm {

constexpr int kMaxD = 8192;
constexpr int kE = 8;                  // elements of a row per thread
constexpr int kRedMost = 8;            // sums of one reduction

template <int TPR>
struct Shape {
  static constexpr int NT = TPR > 256 ? TPR : 256;   // threads per block
  static constexpr int GROUPS = NT / TPR;            // rows side by side in a block
  static constexpr int FWD_ROWS = TPR > 256 ? 1 : 4;   // rows per thread and step
  static constexpr int BWD_ROWS = TPR > 256 ? 1 : 2;
  // Blocks that share an SM: the registers of the rows on their way set it.
  // A long call's grid is just those (d = 128, bf16, 1,048,576 rows forward:
  // 2 a SM with 4 rows a thread 91 us, 3 with 2 rows 95, 4 with 2 rows 97, 3
  // with 4 rows 126, where the third spills; 524,288 rows backward: 2 a SM
  // with 2 rows 81 us, 3 with 1 row 94, 3 with 2 rows 121).
  static constexpr int PER_SM = TPR > 256 ? 1 : 2;
  // forward grid per SM: rows of a whole block are few, more blocks even out
  static constexpr int FWD_GRID = TPR > 256 ? 4 : 2;
};

template <int TPR, bool VEC>
__device__ __forceinline__ int col_of(int lane, int e) {
  return VEC ? lane * kE + e : e * TPR + lane;
}

// A thread's elements of a row as they lie in memory, so that the next rows
// can be fetched while these are worked on, and a bf16 row takes 4 registers.
// Aligned to the 16-byte pieces that it is filled by.
template <int TPR, bool VEC, typename T>
struct Raw {
  alignas(16) T e[kE];
  __device__ __forceinline__ void load(const T *row, int lane, int d, bool live) {
    if constexpr (VEC) {
      constexpr int NV = kE * sizeof(T) / 16;
      uint4 *w = reinterpret_cast<uint4 *>(e);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        w[i] = live && lane * kE < d ? reinterpret_cast<const uint4 *>(row + lane * kE)[i]
                                     : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const int c = i * TPR + lane;
        e[i] = live && c < d ? row[c] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[kE]) const {
#pragma unroll
    for (int i = 0; i < kE; ++i) f[i] = to_f32(e[i]);
  }
};

template <int TPR, bool VEC, typename T>
__device__ __forceinline__ void store_row(T *row, int lane, int d, const float (&f)[kE]) {
  if constexpr (VEC) {
    if (lane * kE < d) {
      if constexpr (sizeof(T) == 2) {
        alignas(16) __nv_bfloat162 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(row + lane * kE) = *reinterpret_cast<const uint4 *>(p);
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

// Sums of NV values over the 32 lanes: halves of the values change places with
// halves of the warp, so that a shuffle sums as many values as there are left
// (9 shuffles for 6 values, not 30).  Returns the sum of value
// warp_value<NV>(lane); the order of the sum is the same for every value.
template <int NV>
constexpr int pow2_values() {
  return NV <= 1 ? 1 : NV <= 2 ? 2 : NV <= 4 ? 4 : 8;
}
template <int NV>
__device__ __forceinline__ int warp_value(int lane) {
  return lane / (32 / pow2_values<NV>());
}
template <int NV>
__device__ __forceinline__ float warp_sums(const float (&v)[NV], int lane) {
  constexpr int P = pow2_values<NV>();
  float t[P];
#pragma unroll
  for (int i = 0; i < P; ++i) t[i] = i < NV ? v[i < NV ? i : 0] : 0.f;
  int o = 16;
#pragma unroll
  for (int n = P / 2; n > 0; n >>= 1, o >>= 1) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = lane & o ? t[i] : t[i + n];
      t[i] = (lane & o ? t[i + n] : t[i]) + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
  return t[0];
}

// Sums of NV values over the TPR threads of each row; every thread gets them.
// With TPR > 32 all threads of the block take part (red: two halves of
// NT / 32 x 8 floats, `turn` alternates them, so one barrier a call is
// enough: a half is written again two calls later, behind the next barrier).
template <int TPR, int NV>
__device__ __forceinline__ void row_sums(float (&v)[NV], float *red, int &turn) {
  const int lane = threadIdx.x & 31;
  if constexpr (TPR < 32) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  } else if constexpr (TPR == 32) {
    const float s = warp_sums(v, lane);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * (32 / pow2_values<NV>()));
  } else {
    constexpr int NW = Shape<TPR>::NT / 32, WPR = TPR / 32;
    const int warp = threadIdx.x >> 5, mine = warp_value<NV>(lane);
    static_assert(NV <= kRedMost, "a half of red holds kRedMost values a warp");
    float *r = red + turn * NW * kRedMost;
    turn ^= 1;
    const float t = warp_sums(v, lane);
    if (lane % (32 / pow2_values<NV>()) == 0 && mine < NV) r[warp * NV + mine] = t;
    __syncthreads();
    const int w0 = warp / WPR * WPR;
    // a lane to a warp's sum of a value, 32 / WPR values at a time
    constexpr int AT_ONCE = 32 / WPR;
#pragma unroll
    for (int i0 = 0; i0 < NV; i0 += AT_ONCE) {
      const int i = i0 + lane / WPR;
      float s = i < NV ? r[(w0 + lane % WPR) * NV + i] : 0.f;
#pragma unroll
      for (int o = WPR / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
      for (int j = 0; j < AT_ONCE; ++j)
        if (i0 + j < NV) v[i0 + j] = __shfl_sync(0xffffffffu, s, j * WPR);
    }
  }
}

template <int TPR>
constexpr int red_floats() {
  return TPR > 32 ? 2 * (Shape<TPR>::NT / 32) * kRedMost : 1;
}

// x becomes x - m (0 in columns past d)
template <int TPR, bool VEC, int ROWS>
__device__ __forceinline__ void centre(float (&x)[ROWS][kE], int lane, int d, float inv_d, bool rms,
                                       float *red, int &turn) {
  if (rms) return;
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

// Rows r0 + r GROUPS + grp of a block's step; the loops of both kernels: the
// next step's rows are on their way while this one's are worked on.
template <int TPR, bool VEC, typename T>
__global__ void __launch_bounds__(Shape<TPR>::NT, Shape<TPR>::PER_SM) norm_fwd_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
    T *__restrict__ out, long rows, int d, float inv_d, float eps, bool rms) {
  constexpr int ROWS = Shape<TPR>::FWD_ROWS, GROUPS = Shape<TPR>::GROUPS;
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
  long r0 = static_cast<long>(blockIdx.x) * GROUPS * ROWS;
  Raw<TPR, VEC, T> next[ROWS];
  auto fetch = [&](long r0) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      next[r].load(x + row * d, lane, d, row < rows);
    }
  };
  fetch(r0);
  for (; r0 < rows; r0 += step) {
    float f[ROWS][kE], s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) next[r].get(f[r]);
    fetch(r0 + step);
    centre<TPR, VEC, ROWS>(f, lane, d, inv_d, rms, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) s[r] = fmaf(f[r][e], f[r][e], s[r]);
    }
    row_sums<TPR, ROWS>(s, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      if (row >= rows) continue;
      const float rstd = 1.f / sqrtf(fmaf(s[r], inv_d, eps));
#pragma unroll
      for (int e = 0; e < kE; ++e) f[r][e] = fmaf(f[r][e] * rstd, fw[e], fb[e]);
      store_row<TPR, VEC>(out + row * d, lane, d, f[r]);
    }
  }
}

// part: [blocks][2][d] partial rows of dw and db (NULL when neither is wanted)
template <int TPR, bool VEC, typename T>
__global__ void __launch_bounds__(Shape<TPR>::NT, Shape<TPR>::PER_SM) norm_bwd_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const T *__restrict__ dy,
    T *__restrict__ dx, float *__restrict__ part, long rows, int d, float inv_d, float eps,
    bool rms) {
  constexpr int ROWS = Shape<TPR>::BWD_ROWS, GROUPS = Shape<TPR>::GROUPS;
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
  long r0 = static_cast<long>(blockIdx.x) * GROUPS * ROWS;
  Raw<TPR, VEC, T> next_x[ROWS], next_y[ROWS];
  auto fetch = [&](long r0) {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      next_x[r].load(x + row * d, lane, d, row < rows);
      next_y[r].load(dy + row * d, lane, d, row < rows);
    }
  };
  fetch(r0);
  for (; r0 < rows; r0 += step) {
    float f[ROWS][kE], s[3 * ROWS];
    Raw<TPR, VEC, T> cur_y[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      next_x[r].get(f[r]);
      cur_y[r] = next_y[r];
    }
    fetch(r0 + step);
    centre<TPR, VEC, ROWS>(f, lane, d, inv_d, rms, red, turn);
    // with c = x - m: sums of c^2, w dy and w dy c, in one reduction
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      s[3 * r] = s[3 * r + 1] = s[3 * r + 2] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float wy = to_f32(cur_y[r].e[e]) * fw[e];
        s[3 * r] = fmaf(f[r][e], f[r][e], s[3 * r]);
        s[3 * r + 1] += wy;
        s[3 * r + 2] = fmaf(wy, f[r][e], s[3 * r + 2]);
      }
    }
    row_sums<TPR, 3 * ROWS>(s, red, turn);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const long row = r0 + r * GROUPS + grp;
      if (row >= rows) continue;   // no row: 1 / sqrt(0 + eps) may be infinite
      const float rstd = 1.f / sqrtf(fmaf(s[3 * r], inv_d, eps));
      const float m0 = rms ? 0.f : s[3 * r + 1] * inv_d;
      const float m1 = s[3 * r + 2] * inv_d * rstd * rstd;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float gy = to_f32(cur_y[r].e[e]);
        aw[e] = fmaf(gy, f[r][e] * rstd, aw[e]);
        ab[e] += gy;
        f[r][e] = rstd * (fmaf(gy, fw[e], -m0) - f[r][e] * m1);
      }
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
// column, each adding every 32nd partial row.  part is written while this grid
// starts, so it is no __restrict__ input: those may be read through a cache
// that takes them as constant for the whole kernel.
__global__ void __launch_bounds__(1024) norm_bwd_sum_kernel(const float *part, float *dw, float *db,
                                                             int blocks, int d) {
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float *dst = blockIdx.y ? db : dw;
  if (!dst) return;
  grid_dependency_wait();   // launched while the partial rows were being made
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int i = ty; i < blocks; i += 32)
      s += part[(static_cast<long>(i) * 2 + blockIdx.y) * d + c];
  red[ty][tx] = s;
  __syncthreads();
  s = warp_sum(red[tx][ty]);
  if (tx == 0 && blockIdx.x * 32 + ty < d) dst[blockIdx.x * 32 + ty] = s;
}

}  // namespace norm
}  // namespace linattn
