// The gated delta rule on CUDA cores, fp32 arithmetic throughout.
//
// A fast weight S [dk, dv] per head that writes what it does not yet return:
//   r_i = v_i - a_i S_{i-1}^T k_i,   u_i = beta_i r_i,   a_i = exp(g_i)
//   S_i = a_i S_{i-1} + k_i u_i^T,   o_i = S_i^T q_i
// and, with D'_i the gradient reaching S_i from the tokens after i,
//   D_i = D'_i + q_i do_i^T,  du_i = D_i^T k_i,  dv_i = beta_i du_i,  dbeta_i = du_i . r_i
//   D'_{i-1} = a_i (D_i - k_i (beta_i du_i)^T)
//   dq_i = S_i do_i,   dk_i = D_i u_i - beta_i a_i S_{i-1} du_i.
// Both recurrences treat the columns of S (the dv axis) independently, so one
// warp carries 8 columns, 4 lanes to a column, or 16 and 2, a lane's dk / 4 or
// dk / 2 rows in its registers, and no two warps wait for each other inside a
// tile of tokens.
// a, rounded to fp32, may be off by 2^-25 a token, and by the same at every token
// of one slow gate: N 2^-25 of the state in the end, where the roundings of S add
// up to sqrt(N) 2^-24.  So the state gets back after every tile of 32 tokens what the
// roundings of its a took.  (Decaying by S + (a - 1) S does the same, but leaves a
// small a no more exact than 2^-25 of one.)
// From the state before the token S^T k and S^T q come out of one pass:
//   o_i = a_i S_{i-1}^T q_i + (k_i . q_i) u_i,
// so a token costs one reduction over the lanes.  What bounds the kernels is a
// warp's own pace: 50 to 100 instructions a token, each after the one it needs
// (2.8 cycles an instruction; issue slots and shared memory half idle).  Two
// tokens to a reduction, S_0^T k_1 = a_0 S^T k_1 + (k_1 . k_0) u_0, were no
// faster (107 ns a token for 112 at dk = 32): fewer waits, more instructions.
//
// The backward runs the forward recurrence once more, keeping r and the state
// at every kSimtChunk tokens, and beside it the reverse recurrence, keeping du
// and D' at the same places, then all chunks at once (delta_bwd_grad_simt_kernel).
#pragma once
#include "common.cuh"
#include "sm100.cuh"

namespace linattn {
namespace delta {

constexpr int kSimtTile = 32;          // tokens staged in shared memory
constexpr int kSimtThreads = 128;      // of a block of the recurrences, at most
constexpr int kSimtChunk = 32;         // tokens between two kept states
// Gates are clamped from below here where they are summed: exp(-128) is 0 in
// fp32, and sums of finite gates stay free of inf - inf.
constexpr float kGateFloor = -128.f;
__device__ __forceinline__ float gate_floor(float g) { return g < kGateFloor ? kGateFloor : g; }

__device__ __forceinline__ void copy_async_16(void *dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_async_4(void *dst, const void *src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}

// Four elements of a row in shared memory as two packed pairs.
__device__ __forceinline__ void load4(const float *p, float2 &a, float2 &b) {
  const float4 x = *reinterpret_cast<const float4 *>(p);
  a = make_float2(x.x, x.y);
  b = make_float2(x.z, x.w);
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float2 &a, float2 &b) {
  const uint2 x = *reinterpret_cast<const uint2 *>(p);
  a = make_float2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
  b = make_float2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Two tiles of tokens in shared memory as they lie in global memory: one that
// the recurrence works on, one on its way while it does.  A tile brought in
// only once the one before was done cost about as much as its 32 tokens.
template <int DK, typename T>
struct SimtTile {
  static constexpr int PER = 16 / sizeof(T);       // elements of a 16-byte piece
  // token t lies in row t + 1: the recurrences fetch one row past either end of
  // a tile, and use it not
  static constexpr int ROWS = kSimtTile + 2;
  T q[2][ROWS][DK], k[2][ROWS][DK], v[2][ROWS][64];
  float4 w[ROWS];                                  // a, a beta, beta, k . q
  float g[2][kSimtTile], b[2][kSimtTile];
  alignas(16) int lost[4];                         // by the roundings of a, a warp each: 2^-40

  // Start the copies of n tokens from tok0; rows past them become zeros.
  __device__ __forceinline__ void stage(int buf, const T *gq, const T *gk, const T *gv,
                                        const float *gate, const float *beta, long tok0, int n,
                                        int dv, int col0, int ncol) {
    const int tid = threadIdx.x, nt = blockDim.x, vc = ncol / PER;
    for (int i = tid; i < kSimtTile * DK / PER; i += nt) {
      const int t = i / (DK / PER), e = (i % (DK / PER)) * PER;
      const long at = (tok0 + (t < n ? t : 0)) * DK + e;
      copy_async_16(&q[buf][t + 1][e], gq + at, t < n);
      copy_async_16(&k[buf][t + 1][e], gk + at, t < n);
    }
    for (int i = tid; i < kSimtTile * vc; i += nt) {
      const int t = i / vc, e = (i % vc) * PER;
      copy_async_16(&v[buf][t + 1][e], gv + (tok0 + (t < n ? t : 0)) * dv + col0 + e, t < n);
    }
    if (tid < kSimtTile) {
      const long at = tok0 + (tid < n ? tid : 0);
      copy_async_4(&b[buf][tid], beta + at, tid < n);
      if (gate) copy_async_4(&g[buf][tid], gate + at, tid < n);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Wait for the tile under way; afterwards no thread works on the other one.
  __device__ __forceinline__ void arrive() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
  }

  // The scalars w of the tile's tokens, blockDim / 32 lanes a token.  Ends with
  // a barrier.
  __device__ __forceinline__ void scalars(int buf, bool gated) {
    const int per = blockDim.x / kSimtTile, t = threadIdx.x / per, p = threadIdx.x % per;
    // from a half on a is 1 + (a - 1), and its rounding known exactly; behind a
    // smaller one there is little left to add up
    const float gate = gated ? g[buf][t] : 0.f, less = expm1f(gate);
    const bool near = fabsf(less) < 0.5f;
    const float a = near ? 1.f + less : expf(gate);
    const int off = near && p == 0 ? __float2int_rn((less - (a - 1.f)) * 0x1p40f) : 0;
    const int sum = __reduce_add_sync(0xffffffffu, off);
    float2 s0 = {}, s1 = {};
    for (int i = p; i < DK / 4; i += per) {
      const int e = 4 * ((i + t * per) & (DK / 4 - 1));   // tokens start in other banks
      float2 q0, q1, k0, k1;
      load4(&q[buf][t + 1][e], q0, q1);
      load4(&k[buf][t + 1][e], k0, k1);
      s0 = ffma2(q0, k0, s0);
      s1 = ffma2(q1, k1, s1);
    }
    float s = (s0.x + s0.y) + (s1.x + s1.y);
    for (int o = per >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) lost[threadIdx.x >> 5] = sum;
    if (p == 0) w[t + 1] = make_float4(a, a * b[buf][t], b[buf][t], s);
    __syncthreads();
  }

  // Before the first tile: warps that the block does not have lose nothing.
  __device__ __forceinline__ void start() {
    if (threadIdx.x < 4) lost[threadIdx.x] = 0;
  }

  // What the tile's a left out of the state, relative to it.
  __device__ __forceinline__ float drift() const {
    const int4 n = *reinterpret_cast<const int4 *>(lost);
    return static_cast<float>((n.x + n.y) + (n.z + n.w)) * 0x1p-40f;
  }
};

// L lanes to a column of S: columns to a warp and pairs of rows to a lane.  With
// L = 2 a token costs the fewest instructions a column; with L = 4 it is done
// sooner where every scheduler of an SM has one warp at most (dk = 64: 132 ns
// against 170 ns a token, fp32), not where it has two (177 ns against 172 ns).
template <int DK, int L>
struct SimtLanes {
  static constexpr int COLS = 32 / L, R2 = DK / (2 * L);
};

// elements 4 L m + 4 rg .. + 3 of a row of the tile for lane group rg: the
// groups read 4 L consecutive elements
template <int DK, int L, typename T>
__device__ __forceinline__ void simt_rows(const T *row, int rg, float2 (&f)[SimtLanes<DK, L>::R2]) {
#pragma unroll
  for (int m = 0; m < SimtLanes<DK, L>::R2 / 2; ++m)
    load4(row + 4 * L * m + 4 * rg, f[2 * m], f[2 * m + 1]);
}

// The lanes' parts of x . y, summed over the lane groups of COLS lanes.
template <int COLS, int R2>
__device__ __forceinline__ float simt_dot(const float2 (&x)[R2], const float2 (&y)[R2]) {
  constexpr int A = R2 < 4 ? R2 : 4;
  float2 p[A] = {};
#pragma unroll
  for (int j = 0; j < R2; ++j) p[j % A] = ffma2(x[j], y[j], p[j % A]);
#pragma unroll
  for (int w = A / 2; w; w >>= 1) {
#pragma unroll
    for (int j = 0; j < w; ++j) p[j] = fadd2(p[j], p[j + w]);
  }
  float s = p[0].x + p[0].y;
#pragma unroll
  for (int o = COLS; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// A lane's rows of one column of a [DK, dv] state: x[j] holds rows
// 4 L (j / 2) + 4 rg + 2 (j % 2) and the one after.
template <int DK, int L>
__device__ __forceinline__ void simt_state_in(float2 (&x)[SimtLanes<DK, L>::R2], const float *src,
                                              int rg, int dv) {
#pragma unroll
  for (int j = 0; j < SimtLanes<DK, L>::R2; ++j) {
    const long at = static_cast<long>(4 * L * (j >> 1) + 4 * rg + 2 * (j & 1)) * dv;
    x[j] = src ? make_float2(src[at], src[at + dv]) : make_float2(0.f, 0.f);
  }
}
template <int DK, int L>
__device__ __forceinline__ void simt_state_out(const float2 (&x)[SimtLanes<DK, L>::R2], float *dst,
                                               int rg, int dv) {
#pragma unroll
  for (int j = 0; j < SimtLanes<DK, L>::R2; ++j) {
    const long at = static_cast<long>(4 * L * (j >> 1) + 4 * rg + 2 * (j & 1)) * dv;
    dst[at] = x[j].x;
    dst[at + dv] = x[j].y;
  }
}

// What a walk through chunks [c0, c1) leaves: the outputs; the state before every
// chunk and every r; only the state at the end (S_out in every mode); or only
// that, from the unit matrix and with v = 0: the chunks' transition.
enum SimtMode { kSimtOut, kSimtKeep, kSimtState, kSimtUnit };

// Forward recurrence of one head from S_in (NULL: zero).  grid (.., dv / columns
// of a block), dk / columns for a transition.  A token's q and k rows are in registers
// before the token before is done, and so are its scalars: their way through
// shared memory is off the chain, and so are a S and beta v.  All lanes compute
// what one lane group stores, so that the warp does not part for it.
template <int DK, int L, typename T, SimtMode MODE>
__device__ __forceinline__ void simt_forward(
    SimtTile<DK, T> &sm, long head, const T *q, const T *k, const T *v, const float *g,
    const float *beta, const float *S_in, T *out, float *S_out, float *keep_S, float *keep_r,
    int N, int dv, int c0, int c1) {
  constexpr int R2 = SimtLanes<DK, L>::R2, COLS = SimtLanes<DK, L>::COLS;
  static_assert(kSimtTile == kSimtChunk, "S is kept once a tile");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rg = lane / COLS;
  const int ncol = COLS * (blockDim.x >> 5), col0 = blockIdx.y * ncol;
  const int lc = COLS * warp + lane % COLS, col = col0 + lc;
  const long base = head * N, plane = static_cast<long>(DK) * dv;
  const int nch = (N + kSimtChunk - 1) / kSimtChunk;
  auto stage = [&](int c) {
    const int t0 = c * kSimtTile;
    sm.stage(c & 1, q, k, v, g, beta, base + t0, min(kSimtTile, N - t0), dv, col0,
             MODE == kSimtUnit ? 0 : ncol);
  };
  sm.start();
  stage(c0);
  float2 S[R2];
  const long first = (base + static_cast<long>(c0) * kSimtTile) * dv + col;
  if constexpr (MODE == kSimtKeep) keep_r += first;
  if constexpr (MODE == kSimtOut) out += first;
  if constexpr (MODE == kSimtUnit) {
#pragma unroll
    for (int j = 0; j < R2; ++j) {
      const int row = 4 * L * (j >> 1) + 4 * rg + 2 * (j & 1);
      S[j] = make_float2(row == col ? 1.f : 0.f, row + 1 == col ? 1.f : 0.f);
    }
  } else {
    simt_state_in<DK, L>(S, S_in ? S_in + col : nullptr, rg, dv);
  }

  for (int c = c0; c < c1; ++c) {
    const int buf = c & 1, n = min(kSimtTile, N - c * kSimtTile);
    sm.arrive();
    if (c + 1 < c1) stage(c + 1);
    sm.scalars(buf, g != nullptr);
    const float drift = sm.drift();
    if constexpr (MODE == kSimtKeep)
      simt_state_out<DK, L>(S, keep_S + (head * nch + c) * plane + col, rg, dv);
    float2 kk[R2], qq[R2];
    simt_rows<DK, L>(sm.k[buf][1], rg, kk);
    simt_rows<DK, L>(sm.q[buf][1], rg, qq);
    float4 w = sm.w[1];
    T x = sm.v[buf][1][lc];
#pragma unroll 4
    for (int t = 0; t < n; ++t) {
      float2 kn[R2], qn[R2];
      simt_rows<DK, L>(sm.k[buf][t + 2], rg, kn);
      simt_rows<DK, L>(sm.q[buf][t + 2], rg, qn);
      const float4 wn = sm.w[t + 2];
      const T xn = sm.v[buf][t + 2][lc];
      const float a = w.x, vt = MODE == kSimtUnit ? 0.f : to_float(x);
      const float ps = simt_dot<COLS>(S, kk), os = simt_dot<COLS>(S, qq);
      const float u = fmaf(-w.y, ps, w.z * vt);
#pragma unroll
      for (int j = 0; j < R2; ++j) {
        S[j] = ffma2(kk[j], make_float2(u, u), fmul2(make_float2(a, a), S[j]));
        kk[j] = kn[j];
        qq[j] = qn[j];
      }
      if constexpr (MODE == kSimtKeep) {
        const float r = fmaf(-a, ps, vt);
        if (rg == 0) *keep_r = r;
        keep_r += dv;
      } else if constexpr (MODE == kSimtOut) {
        const T o = from_f32<T>(fmaf(w.w, u, a * os));
        if (rg == 0) *out = o;
        out += dv;
      }
      w = wn;
      x = xn;
    }
#pragma unroll
    for (int j = 0; j < R2; ++j) S[j] = ffma2(make_float2(drift, drift), S[j], S[j]);
  }
  if constexpr (MODE == kSimtUnit) {
    if (col < DK) simt_state_out<DK, L>(S, S_out + col, rg, DK);
  } else if (S_out) {
    simt_state_out<DK, L>(S, S_out + col, rg, dv);
  }
}

// Reverse recurrence of one head through chunks [c0, c1) from D_in: du of every
// token, D' after every chunk and dv (kSimtKeep), and D' at the start.
template <int DK, int L, typename T, SimtMode MODE>
__device__ __forceinline__ void simt_reverse(
    SimtTile<DK, T> &sm, long head, const T *q, const T *k, const T *dout, const float *g,
    const float *beta, const float *D_in, T *dv_out, float *D_out, float *keep_D,
    float *keep_du, int N, int dv, int c0, int c1) {
  constexpr int R2 = SimtLanes<DK, L>::R2, COLS = SimtLanes<DK, L>::COLS;
  static_assert(kSimtTile == kSimtChunk, "D' is kept once a tile");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rg = lane / COLS;
  const int ncol = COLS * (blockDim.x >> 5), col0 = blockIdx.y * ncol;
  const int lc = COLS * warp + lane % COLS, col = col0 + lc;
  const long base = head * N, plane = static_cast<long>(DK) * dv;
  const int nch = (N + kSimtChunk - 1) / kSimtChunk;
  auto stage = [&](int c) {
    const int t0 = c * kSimtTile;
    sm.stage(c & 1, q, k, dout, g, beta, base + t0, min(kSimtTile, N - t0), dv, col0, ncol);
  };
  sm.start();
  stage(c1 - 1);
  float2 D[R2];
  const long last = (base + min(static_cast<long>(c1) * kSimtTile, static_cast<long>(N)) - 1) * dv + col;
  if constexpr (MODE == kSimtKeep) {
    keep_du += last;
    dv_out += last;
  }
  simt_state_in<DK, L>(D, D_in ? D_in + col : nullptr, rg, dv);

  for (int c = c1 - 1; c >= c0; --c) {
    const int buf = c & 1, n = min(kSimtTile, N - c * kSimtTile);
    sm.arrive();
    if (c > c0) stage(c - 1);
    sm.scalars(buf, g != nullptr);
    const float drift = sm.drift();
    if constexpr (MODE == kSimtKeep)
      simt_state_out<DK, L>(D, keep_D + (head * nch + c) * plane + col, rg, dv);
    float2 kk[R2], qq[R2];
    simt_rows<DK, L>(sm.k[buf][n], rg, kk);
    simt_rows<DK, L>(sm.q[buf][n], rg, qq);
    float4 w = sm.w[n];
    T x = sm.v[buf][n][lc];
#pragma unroll 4
    for (int t = n - 1; t >= 0; --t) {
      float2 kn[R2], qn[R2];
      simt_rows<DK, L>(sm.k[buf][t], rg, kn);
      simt_rows<DK, L>(sm.q[buf][t], rg, qn);
      const float4 wn = sm.w[t];
      const T xn = sm.v[buf][t][lc];
      const float a = w.x, go = to_float(x), from_o = w.w * go, ago = a * go;
      const float ps = simt_dot<COLS>(D, kk);
      const float y = -fmaf(w.y, ps, w.y * from_o);    // -a beta du
#pragma unroll
      for (int j = 0; j < R2; ++j) {
        const float2 d = ffma2(qq[j], make_float2(ago, ago), fmul2(make_float2(a, a), D[j]));
        D[j] = ffma2(kk[j], make_float2(y, y), d);
        kk[j] = kn[j];
        qq[j] = qn[j];
      }
      if constexpr (MODE == kSimtKeep) {
        const float du = ps + from_o;
        const T dvt = from_f32<T>(w.z * du);
        if (rg == 0) {
          *keep_du = du;
          *dv_out = dvt;
        }
        keep_du -= dv;
        dv_out -= dv;
      }
      w = wn;
      x = xn;
    }
#pragma unroll
    for (int j = 0; j < R2; ++j) D[j] = ffma2(make_float2(drift, drift), D[j], D[j]);
  }
  if (D_out) simt_state_out<DK, L>(D, D_out + col, rg, dv);
}

template <int DK, int L, typename T>
__global__ void __launch_bounds__(kSimtThreads) delta_fwd_simt_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const float *__restrict__ g, const float *__restrict__ beta, const float *__restrict__ S_init,
    T *__restrict__ out, float *__restrict__ S_final, int N, int dv) {
  extern __shared__ __align__(16) uint8_t raw[];
  auto &sm = *reinterpret_cast<SimtTile<DK, T> *>(raw);
  const long head = blockIdx.x, state = head * DK * dv;
  simt_forward<DK, L, T, kSimtOut>(sm, head, q, k, v, g, beta, S_init ? S_init + state : nullptr,
                                   out, S_final ? S_final + state : nullptr, nullptr, nullptr, N,
                                   dv, 0, (N + kSimtChunk - 1) / kSimtChunk);
}

// Few heads: both recurrences go through `segs` segments of `len` chunks side by
// side.  A segment maps the state before it, S -> M S + B, and the gradient after
// it, D -> M^T D + E.  One launch forms B (from zero; from S_init in the first
// segment), E (from zero; from dS_final in the last) and M; the next joins them;
// then the segments run from the states between them.
//   S  [segs - 1][BH][DK][dv]   B of segment j, then the state after it
//   D  [segs - 1][BH][DK][dv]   E of segment j + 1, then the gradient before it
//   M  [segs - 2][BH][DK][DK]   of segment j + 1
struct SimtSegments {
  float *S, *D, *M;
  int segs, len;
};

template <int DK, int L, typename T>
__global__ void __launch_bounds__(kSimtThreads) delta_transition_simt_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ dout, const float *__restrict__ g, const float *__restrict__ beta,
    const float *__restrict__ S_init, const float *__restrict__ dS_final, SimtSegments x, int BH,
    int N, int dv) {
  extern __shared__ __align__(16) uint8_t raw[];
  auto &sm = *reinterpret_cast<SimtTile<DK, T> *>(raw);
  const int part = blockIdx.x / BH, col0 = blockIdx.y * (blockDim.x / L);
  const long head = blockIdx.x % BH, state = static_cast<long>(DK) * dv;
  const int nch = (N + kSimtChunk - 1) / kSimtChunk, segs = x.segs;
  if (part < 2 * (segs - 1) ? col0 >= dv : col0 >= DK) return;
  T *none = nullptr;
  if (part < segs - 1) {
    const int j = part;
    simt_forward<DK, L, T, kSimtState>(
        sm, head, q, k, v, g, beta, j == 0 && S_init ? S_init + head * state : nullptr, none,
        x.S + (static_cast<long>(j) * BH + head) * state, nullptr, nullptr, N, dv, j * x.len,
        (j + 1) * x.len);
  } else if (part < 2 * (segs - 1)) {
    const int j = part - (segs - 1) + 1;
    simt_reverse<DK, L, T, kSimtState>(
        sm, head, q, k, dout, g, beta,
        j == segs - 1 && dS_final ? dS_final + head * state : nullptr, none,
        x.D + (static_cast<long>(j - 1) * BH + head) * state, nullptr, nullptr, N, dv, j * x.len,
        min((j + 1) * x.len, nch));
  } else {
    const int j = part - 2 * (segs - 1) + 1;
    simt_forward<DK, L, T, kSimtUnit>(sm, head, q, k, v, g, beta, nullptr, none,
                                      x.M + (static_cast<long>(j - 1) * BH + head) * DK * DK, nullptr,
                                      nullptr, N, dv, j * x.len, (j + 1) * x.len);
  }
}

// S after segment j = M_j S + B_j for j = 1 .. segs - 2, and D before segment j =
// M_j^T D + E_j for j = segs - 2 .. 1: grid (BH, dv / 16, 2), 16 columns a block, a
// thread to a row and DK / 16 of them.  The chain of steps is what the kernel
// waits for: the next M and B are in registers before this step's product.
template <int DK>
constexpr int simt_join_smem() { return (DK * (DK + 1) + DK * 16 + 16) * 4; }

template <int DK>
__global__ void __launch_bounds__(256) delta_join_simt_kernel(SimtSegments x, int BH, int dv) {
  constexpr int P = DK / 16, NV = DK * DK / 4 < 256 ? 1 : DK * DK / 1024, MS = DK + 1;
  extern __shared__ __align__(16) float sm[];
  float *cur = sm, *sM = sm + DK * 16;   // [DK][16], [DK][DK + 1]
  const int tid = threadIdx.x, r = tid % DK, c = tid / DK * P;
  const long head = blockIdx.x, state = static_cast<long>(DK) * dv;
  const bool rev = blockIdx.z != 0;
  float *base = (rev ? x.D : x.S) + static_cast<long>(r) * dv + 16 * blockIdx.y + c;
  auto slot = [&](int j) { return base + (static_cast<long>(j) * BH + head) * state; };
  float4 m[NV];
  float b[P];
  auto fetch = [&](int i) {
    if (i >= x.segs - 1) return;
    const int j = rev ? x.segs - 1 - i : i;
    const float *M = x.M + (static_cast<long>(j - 1) * BH + head) * DK * DK;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (4 * (tid + 256 * n) < DK * DK) m[n] = reinterpret_cast<const float4 *>(M)[tid + 256 * n];
    const float *B = slot(rev ? j - 1 : j);
#pragma unroll
    for (int p = 0; p < P; ++p) b[p] = B[p];
  };
  const float *from = slot(rev ? x.segs - 2 : 0);
#pragma unroll
  for (int p = 0; p < P; ++p) cur[r * 16 + c + p] = from[p];
  fetch(1);
  for (int i = 1; i < x.segs - 1; ++i) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int at = 4 * (tid + 256 * n);
      if (at < DK * DK) {
        float *d = sM + at / DK * MS + at % DK;
        d[0] = m[n].x; d[1] = m[n].y; d[2] = m[n].z; d[3] = m[n].w;
      }
    }
    float acc[P];
#pragma unroll
    for (int p = 0; p < P; ++p) acc[p] = b[p];
    fetch(i + 1);
    __syncthreads();
    const float *row = rev ? sM + r : sM + r * MS;
    const int step = rev ? MS : 1;
#pragma unroll 8
    for (int e = 0; e < DK; ++e) {
      const float y = row[e * step];
#pragma unroll
      for (int p = 0; p < P; ++p) acc[p] = fmaf(y, cur[e * 16 + c + p], acc[p]);
    }
    __syncthreads();
    float *dst = slot(rev ? x.segs - 2 - i : i);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      dst[p] = acc[p];
      cur[r * 16 + c + p] = acc[p];
    }
  }
}

// Both recurrences of the backward, which do not need each other: grid
// (2 segs B H, ..), the segments forwards and then the segments backwards.
// SEGS = false: one segment, whose bounds and pointers need no register of
// their own (256 tokens in fp32, 4 heads of d = 64: 33.6 us, 35.0 with them; 200
// heads of d = 16: 25.6 and 27.7).
template <int DK, int L, typename T, bool SEGS>
__global__ void __launch_bounds__(kSimtThreads) delta_sweep_simt_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
    const T *__restrict__ dout, const float *__restrict__ g, const float *__restrict__ beta,
    const float *__restrict__ S_init, const float *__restrict__ dS_final, T *__restrict__ dv_out,
    float *__restrict__ dS_init, float *__restrict__ keep_S, float *__restrict__ keep_D,
    float *__restrict__ keep_r, float *__restrict__ keep_du, SimtSegments x, int BH, int N, int dv) {
  extern __shared__ __align__(16) uint8_t raw[];
  auto &sm = *reinterpret_cast<SimtTile<DK, T> *>(raw);
  const int segs = SEGS ? x.segs : 1, part = blockIdx.x / BH, j = SEGS ? part % segs : 0;
  const long head = blockIdx.x % BH, state = static_cast<long>(DK) * dv;
  const int nch = (N + kSimtChunk - 1) / kSimtChunk;
  const int c0 = SEGS ? j * x.len : 0, c1 = SEGS ? min(c0 + x.len, nch) : nch;
  if (part < segs) {
    const float *S0 = j ? x.S + static_cast<long>(j - 1) * BH * state : S_init;
    simt_forward<DK, L, T, kSimtKeep>(sm, head, q, k, v, g, beta, S0 ? S0 + head * state : nullptr,
                                      static_cast<T *>(nullptr), nullptr, keep_S, keep_r, N, dv, c0,
                                      c1);
  } else {
    const float *D1 = j < segs - 1 ? x.D + static_cast<long>(j) * BH * state : dS_final;
    simt_reverse<DK, L, T, kSimtKeep>(sm, head, q, k, dout, g, beta,
                                      D1 ? D1 + head * state : nullptr, dv_out,
                                      j == 0 && dS_init ? dS_init + head * state : nullptr, keep_D,
                                      keep_du, N, dv, c0, c1);
  }
}

// The gradients of one chunk of C = 32 tokens, all chunks at once.  With S0
// the state before the chunk, D the gradient after it, gamma the sums of the
// gates in the chunk, Gam_ts = exp(gamma_t - gamma_s), U = beta r, X = beta du:
//   M = Gam o (dO U^T) (s <= t),  Y = Gam o (X U^T) (s < t)
//   dq = e^gamma dO S0^T + M K
//   dk = e^(gamma_C - gamma) U D^T + M^T Q - (Y + Y^T) K - e^gamma X S0^T
//   dbeta = rowsum(du o r)
// dg_i sums what passes token i: pairs t >= i > s of
// E = (Q K^T) o M - (K K^T) o Y, what S0 hands to t >= i, what s < i hands to
// D, and e^gamma_C <S0, D>.  The pairs come as suffix sums of row sums minus
// column sums of the same E, so that pairs on one side of i cancel to a
// rounding of fp32, however small dg_i is beside them.
constexpr int kSimtGradThreads = 256;

template <int DK, int DV>
constexpr int delta_grad_simt_smem_floats() {
  constexpr int C = kSimtChunk;
  return 2 * C * (DK + 1) + 3 * C * (DV + 1) + DK * (DV + 1) + 3 * C * (C + 1) + 10 * C + 16;
}

template <int DK, int DV, typename T>
__global__ void __launch_bounds__(kSimtGradThreads) delta_bwd_grad_simt_kernel(
    const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ dout,
    const float *__restrict__ g, const float *__restrict__ beta, const float *__restrict__ keep_S,
    const float *__restrict__ keep_D, const float *__restrict__ keep_r,
    const float *__restrict__ keep_du, T *__restrict__ dq, T *__restrict__ dk,
    float *__restrict__ dg, float *__restrict__ dbeta, int N, int nch) {
  constexpr int C = kSimtChunk, NT = kSimtGradThreads, QS = DK + 1, VS = DV + 1, AS = C + 1;
  constexpr int RC = C / 16, NK = DK / 16;
  extern __shared__ __align__(16) float sm[];
  float *sQ = sm;                  // [C][DK+1]
  float *sK = sQ + C * QS;         // [C][DK+1]
  float *sG = sK + C * QS;         // [C][DV+1] dout
  float *sU = sG + C * VS;         // [C][DV+1] u = beta r
  float *sX = sU + C * VS;         // [C][DV+1] beta du
  float *sS = sX + C * VS;         // [DK][DV+1] S0, then D
  float *sM = sS + DK * VS;        // [C][C+1]
  float *sY = sM + C * AS;         // [C][C+1]
  float *sE = sY + C * AS;         // [C][C+1]
  float *hi = sE + C * AS;         // [C] gamma, high and low parts
  float *lo = hi + C;
  float *eg = lo + C;              // [C] exp(gamma_t)
  float *el = eg + C;              // [C] exp(gamma_C - gamma_t)
  float *sa = el + C;              // [C] what S0 hands to token t
  float *sb = sa + C;              // [C] what token s hands to D
  float *se = sb + C;              // [C] row sum minus column sum of E
  float *red = se + C;             // [8 + 1]

  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const long head = blockIdx.x / nch;
  const int c = static_cast<int>(blockIdx.x % nch);
  const int c0 = c * C, Cv = min(C, N - c0);
  const long tok = head * N + c0;

  for (int i = tid; i < C * DK / 8; i += NT) {
    const int t = i / (DK / 8), e = (i % (DK / 8)) * 8;
    float f[8] = {}, h[8] = {};
    if (t < Cv) {
      load8_f32(q + (tok + t) * DK + e, f);
      load8_f32(k + (tok + t) * DK + e, h);
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      sQ[t * QS + e + x] = f[x];
      sK[t * QS + e + x] = h[x];
    }
  }
  for (int t = tid >> 3; t < C; t += NT / 8) {   // 8 threads a token: dbeta = du . r
    float s = 0.f;
    const float b = t < Cv ? beta[tok + t] : 0.f;
    for (int e = (tid & 7) * 8; e < DV; e += 64) {
      float f[8] = {}, r[8] = {}, u[8] = {};
      if (t < Cv) {
        load8_f32(dout + (tok + t) * DV + e, f);
        load8_f32(keep_r + (tok + t) * DV + e, r);
        load8_f32(keep_du + (tok + t) * DV + e, u);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        sG[t * VS + e + x] = f[x];
        sU[t * VS + e + x] = b * r[x];
        sX[t * VS + e + x] = b * u[x];
        s = fmaf(r[x], u[x], s);
      }
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((tid & 7) == 0 && t < Cv) dbeta[tok + t] = s;
  }
  if (tid < 32) {
    double x = tid < Cv && g ? static_cast<double>(gate_floor(g[tok + tid])) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (tid >= o) x += y;
    }
    const double last = __shfl_sync(0xffffffffu, x, 31);
    hi[tid] = static_cast<float>(x);
    lo[tid] = static_cast<float>(x - static_cast<double>(static_cast<float>(x)));
    eg[tid] = expf(static_cast<float>(x));
    el[tid] = expf(static_cast<float>(last - x));
  }
  const float *S0 = keep_S + (head * nch + c) * DK * DV, *D = keep_D + (head * nch + c) * DK * DV;
  auto load_state = [&](const float *src) {
    for (int i = tid; i < DK * DV / 4; i += NT) {
      const float4 x = reinterpret_cast<const float4 *>(src)[i];
      float *d = sS + (4 * i / DV) * VS + (4 * i) % DV;
      d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
    }
  };
  load_state(S0);
  __syncthreads();
  auto gam = [&](int t, int s) { return expf((hi[t] - hi[s]) + (lo[t] - lo[s])); };

  // M, Y and E
  {
    float a1[RC][RC] = {}, a2[RC][RC] = {}, b1[RC][RC] = {}, b2[RC][RC] = {};
#pragma unroll 2
    for (int a = 0; a < DK; ++a) {
#pragma unroll
      for (int i = 0; i < RC; ++i)
#pragma unroll
        for (int m = 0; m < RC; ++m) {
          const float y = sK[(tx + 16 * m) * QS + a];
          a1[i][m] = fmaf(sQ[(ty + 16 * i) * QS + a], y, a1[i][m]);
          a2[i][m] = fmaf(sK[(ty + 16 * i) * QS + a], y, a2[i][m]);
        }
    }
#pragma unroll 2
    for (int a = 0; a < DV; ++a) {
#pragma unroll
      for (int i = 0; i < RC; ++i)
#pragma unroll
        for (int m = 0; m < RC; ++m) {
          const float y = sU[(tx + 16 * m) * VS + a];
          b1[i][m] = fmaf(sG[(ty + 16 * i) * VS + a], y, b1[i][m]);
          b2[i][m] = fmaf(sX[(ty + 16 * i) * VS + a], y, b2[i][m]);
        }
    }
#pragma unroll
    for (int i = 0; i < RC; ++i)
#pragma unroll
      for (int m = 0; m < RC; ++m) {
        const int t = ty + 16 * i, s = tx + 16 * m;
        const float w = s <= t ? gam(t, s) : 0.f;
        const float mm = w * b1[i][m], yy = s < t ? w * b2[i][m] : 0.f;
        sM[t * AS + s] = mm;
        sY[t * AS + s] = yy;
        sE[t * AS + s] = s < t ? a1[i][m] * mm - a2[i][m] * yy : 0.f;
      }
  }
  __syncthreads();
  if (tid < C) {
    float s = 0.f;
    for (int x = 0; x < tid; ++x) s += sE[tid * AS + x];
    for (int x = tid + 1; x < C; ++x) s -= sE[x * AS + tid];
    se[tid] = s;
  }
  // the products with S0: dq's and the last term of dk; what S0 hands to t
  float dka[RC][NK];
  {
    float x1[RC][NK] = {}, x2[RC][NK] = {};
    for (int a = 0; a < DV; ++a) {
      float y[NK];
#pragma unroll
      for (int m = 0; m < NK; ++m) y[m] = sS[(tx + 16 * m) * VS + a];
#pragma unroll
      for (int i = 0; i < RC; ++i) {
        const float p = sG[(ty + 16 * i) * VS + a], r = sX[(ty + 16 * i) * VS + a];
#pragma unroll
        for (int m = 0; m < NK; ++m) {
          x1[i][m] = fmaf(p, y[m], x1[i][m]);
          x2[i][m] = fmaf(r, y[m], x2[i][m]);
        }
      }
    }
    float x3[RC][NK] = {};
    for (int s = 0; s < C; ++s) {
#pragma unroll
      for (int m = 0; m < NK; ++m) {
        const float y = sK[s * QS + tx + 16 * m];
#pragma unroll
        for (int i = 0; i < RC; ++i) x3[i][m] = fmaf(sM[(ty + 16 * i) * AS + s], y, x3[i][m]);
      }
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      const int t = ty + 16 * i;
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < NK; ++m) {
        const int e = tx + 16 * m;
        const float p = eg[t] * x1[i][m], r = eg[t] * x2[i][m];
        s = fmaf(sQ[t * QS + e], p, s);
        s = fmaf(-sK[t * QS + e], r, s);
        dka[i][m] = -r;
        if (t < Cv) dq[(tok + t) * DK + e] = from_f32<T>(p + x3[i][m]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o, 16);
      if (tx == 0) sa[t] = s;
    }
  }
  // <S0, D>, then D in the place of S0
  float sd = 0.f;
  for (int i = tid; i < DK * DV; i += NT) sd = fmaf(sS[(i / DV) * VS + i % DV], D[i], sd);
  sd = warp_sum(sd);
  if ((tid & 31) == 0) red[tid >> 5] = sd;
  __syncthreads();
  load_state(D);
  __syncthreads();
  {
    float x1[RC][NK] = {}, x2[RC][NK] = {};
    for (int a = 0; a < DV; ++a) {
      float y[NK];
#pragma unroll
      for (int m = 0; m < NK; ++m) y[m] = sS[(tx + 16 * m) * VS + a];
#pragma unroll
      for (int i = 0; i < RC; ++i) {
        const float p = sU[(ty + 16 * i) * VS + a];
#pragma unroll
        for (int m = 0; m < NK; ++m) x1[i][m] = fmaf(p, y[m], x1[i][m]);
      }
    }
    for (int s = 0; s < C; ++s) {
#pragma unroll
      for (int i = 0; i < RC; ++i) {
        const int t = ty + 16 * i;
        const float mt = sM[s * AS + t], yy = sY[t * AS + s] + sY[s * AS + t];
#pragma unroll
        for (int m = 0; m < NK; ++m)
          x2[i][m] = fmaf(mt, sQ[s * QS + tx + 16 * m],
                          fmaf(-yy, sK[s * QS + tx + 16 * m], x2[i][m]));
      }
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      const int t = ty + 16 * i;
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < NK; ++m) {
        const int e = tx + 16 * m;
        const float p = el[t] * x1[i][m];
        s = fmaf(sK[t * QS + e], p, s);
        if (t < Cv) dk[(tok + t) * DK + e] = from_f32<T>(p + x2[i][m] + dka[i][m]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o, 16);
      if (tx == 0) sb[t] = s;
    }
  }
  __syncthreads();
  if (dg && tid < 32) {
    // suffix sums of se + sa, exclusive prefix sums of sb
    float suf = se[tid] + sa[tid], pre = sb[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_down_sync(0xffffffffu, suf, o);
      const float y = __shfl_up_sync(0xffffffffu, pre, o);
      if (tid + o < 32) suf += x;
      if (tid >= o) pre += y;
    }
    pre = __shfl_up_sync(0xffffffffu, pre, 1);
    if (tid == 0) pre = 0.f;
    float all = 0.f;
    for (int w = 0; w < NT / 32; ++w) all += red[w];
    if (tid < Cv) dg[tok + tid] = suf + pre + eg[C - 1] * all;
  }
}

}  // namespace delta
}  // namespace linattn
