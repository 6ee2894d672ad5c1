// Gated layer / RMS norm of rows and its gradients.
//
//   u = x (or x silu(z) with the gate first),  hat = (u - mean) rstd,
//   rstd = (mean((u - mean)^2) + eps)^-1/2  (RMS: mean = 0),
//   out = hat w + b, times silu(z) with the gate last.
// Gradients, dy = dout (times silu(z) with the gate last), dhat = dy w:
//   dw = sum_rows dy hat,  db = sum_rows dy,
//   du = rstd (dhat - mean(dhat) - hat mean(dhat hat))   (RMS: without mean(dhat)),
//   gate last:  dz = dout (hat w + b) silu'(z), dx = du;
//   gate first: dz = du x silu'(z),             dx = du silu(z).
//
// Bound by HBM: a row stays in the registers of TPR threads (NC vectors of VEC elements each)
// from its one load to its store; the variance is taken of the centred row, in fp32. The backward
// forms the row's statistics again from x, which it has to read anyway, so the forward keeps
// nothing for it. Measured: forward 33860 x 32 gated rows of 128, bf16, 155 us (5.4 TB/s);
// gradients of 16384 x 16 such rows 61 us (5.5 TB/s) and 6 for the sums, of 16384 rows of 4096 87
// us (4.9 TB/s) and 9. Gradients of rows above 8192 entries, and of rows above 4096 element by
// element, run out of registers and spill: 8192 rows of 16384, gated, 522 us (2.6 TB/s), of 4097
// 226. A short row takes 8 to 64 threads, so that all loads of a wave are one vector a thread and
// the sums stay in a wave; longer ones a workgroup.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kModeNone = 0, kModeLast = 1, kModeFirst = 2;

struct NormArgs {
  int64_t rows, x_stride, z_stride, dz_stride;
  int heads, dim;
  float eps, inv_dim;
  bool rms;
};

// Sums of A values over the TPR threads of a row (aligned groups; more than a wave: over the
// whole workgroup, through LDS).
template <int TPR, int A>
__device__ __forceinline__ void row_sum(float (&v)[A], float (*s_red)[A]) {
#pragma unroll
  for (int off = 1; off < (TPR < 64 ? TPR : 64); off <<= 1)
#pragma unroll
    for (int i = 0; i < A; ++i) v[i] += __shfl_xor(v[i], off, 64);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    __syncthreads();  // the row before has been read
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < A; ++i) s_red[wv][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < A; ++i) {
      float a = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) a += s_red[k][i];
      v[i] = a;
    }
  }
}

// The threads of a row: vector i of thread l covers columns (i TPR + l) VEC ...
template <int VEC, int TPR, int NC>
struct RowCols {
  int col[NC];
  bool in[NC];
  __device__ __forceinline__ RowCols(int l, int dim) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      col[i] = (i * TPR + l) * VEC;
      in[i] = col[i] < dim;
    }
  }
};

template <typename T, int VEC, int NC>
__device__ __forceinline__ void load_cols(const T* p, const int (&col)[NC], const bool (&in)[NC],
                                          float (&v)[NC][VEC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (in[i]) {
      load_vec<VEC>(p + col[i], v[i]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
    }
  }
}

// The same as they are stored, for rows that wait in registers: with the backward's rows loaded as
// they are and converted at their use 16384 x 16 gated rows of 128 take 71 us a call, not 81.
template <typename T, int VEC, int NC>
__device__ __forceinline__ void load_raw(const T* p, const int (&col)[NC], const bool (&in)[NC],
                                         Raw<T, VEC> (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (in[i])
      v[i].load(p + col[i]);
    else
      v[i].zero();
  }
}
template <typename T, int VEC, int NC>
__device__ __forceinline__ void unpack(const Raw<T, VEC> (&v)[NC], float (&x)[NC][VEC]) {
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[i][e] = v[i][e];
}

// Where a row group's row of a step of the loop is: token, head, and whether it exists.
struct RowAt {
  int64_t row, t, h;
  bool live;
  __device__ __forceinline__ RowAt(int64_t r, const NormArgs& a) : row(r), live(r < a.rows) {
    t = live ? r / a.heads : 0;
    h = live ? r - t * a.heads : 0;
  }
};

// Workgroup threads: at least one row, 256 where rows are narrower.
template <int TPR>
constexpr int kBlock = TPR > 256 ? TPR : 256;

// Mean and reciprocal deviation of the row u.
template <int VEC, int TPR, int NC>
__device__ __forceinline__ void row_stats(const float (&u)[NC][VEC], const bool (&in)[NC],
                                          const NormArgs& a, float (*s_red)[1], float& mean,
                                          float& rstd) {
  mean = 0.f;
  if (!a.rms) {
    float m[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) m[0] += u[i][e];
    row_sum<TPR, 1>(m, s_red);
    mean = m[0] * a.inv_dim;
  }
  float q[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (in[i])
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = u[i][e] - mean;
        q[0] = __builtin_fmaf(d, d, q[0]);
      }
  row_sum<TPR, 1>(q, s_red);
  rstd = 1.f / sqrtf(__builtin_fmaf(q[0], a.inv_dim, a.eps));
}

template <typename T, int VEC, int TPR, int NC, int MODE>
__global__ __launch_bounds__(kBlock<TPR>) void norm_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ z, T* __restrict__ out, NormArgs a) {
  constexpr int RPB = kBlock<TPR> / TPR;  // rows of a workgroup at a time
  __shared__ float s_red[TPR > 64 ? TPR / 64 : 1][1];
  const int l = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const RowCols<VEC, TPR, NC> k(l, a.dim);
  float w[NC][VEC], b[NC][VEC];
  load_cols<float, VEC, NC>(weight, k.col, k.in, w);
  if (bias) load_cols<float, VEC, NC>(bias, k.col, k.in, b);
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += step) {
    // a wider row's threads leave the loop together; a narrow one's past the end do no harm
    const RowAt at(r0 + rg, a);
    bool in[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) in[i] = k.in[i] && at.live;
    float u[NC][VEC], g[NC][VEC];
    load_cols<T, VEC, NC>(x + at.t * a.x_stride + at.h * a.dim, k.col, in, u);
    if constexpr (MODE != kModeNone) {
      load_cols<T, VEC, NC>(z + at.t * a.z_stride + at.h * a.dim, k.col, in, g);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          g[i][e] *= sigmoidf(g[i][e]);
          if constexpr (MODE == kModeFirst) u[i][e] *= g[i][e];
        }
    }
    float mean, rstd;
    row_stats<VEC, TPR, NC>(u, in, a, s_red, mean, rstd);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!in[i]) continue;
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y[e] = (u[i][e] - mean) * rstd * w[i][e];
        if (bias) y[e] += b[i][e];
        if constexpr (MODE == kModeLast) y[e] *= g[i][e];
      }
      store_vec<VEC>(out + at.row * a.dim + k.col[i], y);
    }
  }
}

template <typename T, int VEC, int TPR, int NC, int MODE>
__global__ __launch_bounds__(kBlock<TPR>) void norm_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
    const T* __restrict__ z, const T* __restrict__ dout, T* __restrict__ dx, T* __restrict__ dz,
    float* __restrict__ partial, NormArgs a) {
  constexpr int RPB = kBlock<TPR> / TPR;
  __shared__ float s_one[TPR > 64 ? TPR / 64 : 1][1];
  __shared__ float s_two[TPR > 64 ? TPR / 64 : 1][2];
  const int l = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  const RowCols<VEC, TPR, NC> k(l, a.dim);
  float w[NC][VEC], b[NC][VEC], dw[NC][VEC], db[NC][VEC];
  load_cols<float, VEC, NC>(weight, k.col, k.in, w);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = b[i][e] = 0.f;
  if (bias) load_cols<float, VEC, NC>(bias, k.col, k.in, b);
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += step) {
    const RowAt at(r0 + rg, a);
    const int64_t row = at.row, t = at.t, h = at.h;
    bool in[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) in[i] = k.in[i] && at.live;
    float u[NC][VEC], d[NC][VEC], zz[NC][VEC];
    Raw<T, VEC> xr[NC], dr[NC], zr[NC];
    load_raw<T, VEC, NC>(x + t * a.x_stride + h * a.dim, k.col, in, xr);
    load_raw<T, VEC, NC>(dout + row * (int64_t)a.dim, k.col, in, dr);
    if constexpr (MODE != kModeNone)
      load_raw<T, VEC, NC>(z + t * a.z_stride + h * a.dim, k.col, in, zr);
    unpack<T, VEC, NC>(xr, u);
    unpack<T, VEC, NC>(dr, d);
    if constexpr (MODE != kModeNone) unpack<T, VEC, NC>(zr, zz);
    float xx[MODE == kModeFirst ? NC : 1][VEC];
    if constexpr (MODE == kModeFirst) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xx[i][e] = u[i][e];
          u[i][e] *= zz[i][e] * sigmoidf(zz[i][e]);
        }
    }
    float mean, rstd;
    row_stats<VEC, TPR, NC>(u, in, a, s_one, mean, rstd);
    float sums[2] = {0.f, 0.f};  // of dhat and of dhat hat
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!in[i]) continue;
      float gz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float hat = (u[i][e] - mean) * rstd;
        u[i][e] = hat;
        if constexpr (MODE == kModeLast) {
          const float s = sigmoidf(zz[i][e]);
          const float y = __builtin_fmaf(hat, w[i][e], b[i][e]);
          gz[e] = d[i][e] * y * (s * __builtin_fmaf(zz[i][e], 1.f - s, 1.f));
          d[i][e] *= zz[i][e] * s;
        }
        dw[i][e] = __builtin_fmaf(d[i][e], hat, dw[i][e]);
        db[i][e] += d[i][e];
        d[i][e] *= w[i][e];
        sums[0] += d[i][e];
        sums[1] = __builtin_fmaf(d[i][e], hat, sums[1]);
      }
      if constexpr (MODE == kModeLast)
        store_vec<VEC>(dz + t * a.dz_stride + h * a.dim + k.col[i], gz);
    }
    row_sum<TPR, 2>(sums, s_two);
    const float m0 = a.rms ? 0.f : sums[0] * a.inv_dim, m1 = sums[1] * a.inv_dim;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!in[i]) continue;
      float du[VEC], gz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        du[e] = rstd * (d[i][e] - m0 - u[i][e] * m1);
        if constexpr (MODE == kModeFirst) {
          const float s = sigmoidf(zz[i][e]);
          gz[e] = du[e] * xx[i][e] * (s * __builtin_fmaf(zz[i][e], 1.f - s, 1.f));
          du[e] *= zz[i][e] * s;
        }
      }
      store_vec<VEC>(dx + row * (int64_t)a.dim + k.col[i], du);
      if constexpr (MODE == kModeFirst)
        store_vec<VEC>(dz + t * a.dz_stride + h * a.dim + k.col[i], gz);
    }
  }
  // one partial row per workgroup, the row groups of a workgroup added in a fixed order
  float* const pw = partial + (int64_t)blockIdx.x * 2 * a.dim;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (k.in[i]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          pw[k.col[i] + e] = dw[i][e];
          if (bias) pw[a.dim + k.col[i] + e] = db[i][e];
        }
      }
  } else {
    constexpr int W = TPR * NC * VEC;
    __shared__ float s_part[RPB * W];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (which && !bias) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          s_part[rg * W + (i * TPR + l) * VEC + e] = which ? db[i][e] : dw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < W && c < a.dim; c += kBlock<TPR>) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < RPB; ++r) v += s_part[r * W + c];
        pw[which * a.dim + c] = v;
      }
    }
  }
}

// dweight and dbias from the workgroups' partial rows [blocks][2][dim], added in a fixed order: a
// thread's rows four at a time, then the threads of a column.
constexpr int kSumCols = 16, kSumRows = 64;
__global__ __launch_bounds__(kSumCols * kSumRows) void norm_bwd_sum_kernel(
    const float* __restrict__ partial, int blocks, int dim, float* __restrict__ dweight,
    float* __restrict__ dbias) {
  __shared__ float s_red[kSumRows][kSumCols + 1];
  const int col = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
  const int c = (int)blockIdx.x * kSumCols + col;
  float* const to = blockIdx.y ? dbias : dweight;
  if (!to) return;  // the whole workgroup
  const float* const p = partial + (int64_t)blockIdx.y * dim + c;
  float v = 0.f;
  if (c < dim) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = r; k < blocks; k += 4 * kSumRows)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + i * kSumRows < blocks) a[i] += p[(int64_t)(k + i * kSumRows) * 2 * dim];
    v = (a[0] + a[1]) + (a[2] + a[3]);
  }
  s_red[r][col] = v;
  for (int half = kSumRows / 2; half > 0; half /= 2) {
    __syncthreads();
    if (r < half) s_red[r][col] += s_red[r + half][col];
  }
  if (r == 0 && c < dim) to[c] = s_red[0][col];
}

// Rows handled at a time by one workgroup of the kernel that serves a row length.
struct Pick {
  int tpr, nc;
};
Pick pick(const NormShape& s) {
  const int vec = s.vec ? (s.bf16 ? 8 : 4) : 1;
  const int n = (s.dim + vec - 1) / vec;  // vectors of a row
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  if (n <= 256) return {256, 1};  // more vectors a thread spill in the gated gradients
  if (n <= 512) return {256, 2};
  if (n <= 1024) return {512, 2};
  if (n <= 2048) return {1024, 2};
  if (n <= 4096) return {1024, 4};
  return {1024, 16};  // element by element up to 16384
}

int rows_per_block(const Pick& p) { return p.tpr > 256 ? 1 : 256 / p.tpr; }

// Workgroups of a launch; the rest of the rows in the kernel's loop, which keeps the weights (and
// the gradients' sums) in registers. Forward: the more the better (33860 x 32 rows of 128, gated:
// 154 us with 16384, 161 with 4096; the next row's loads ahead of this row's work took 6 % more).
// Backward: each writes a partial row of dweight and dbias, and 768 are what the device holds
// (us a call with 512, 768 and 1024: 16384 rows of 4096 105, 93 and 103; 16384 x 16 heads of 128 76,
// 71 and 73).
int64_t fwd_blocks(const NormShape& s, const Pick& p) {
  const int64_t all = cdiv(s.N * s.heads, rows_per_block(p));
  return all < 16384 ? all : 16384;
}
int64_t bwd_blocks(const NormShape& s, const Pick& p) {
  const int64_t all = cdiv(s.N * s.heads, rows_per_block(p));
  const int64_t most = p.tpr > 512 ? 256 : p.tpr > 256 ? 512 : 768;
  return all < most ? all : most;
}

NormArgs args_of(const NormShape& s) {
  return NormArgs{s.N * s.heads, s.x_stride, s.z_stride, s.dz_stride, s.heads, s.dim,
                  s.eps, (float)(1.0 / s.dim), s.rms};
}

template <typename T, int VEC, int TPR, int NC>
hipError_t fwd_k(const NormShape& s, int64_t blocks, const void* x, const float* weight,
                 const float* bias, const void* z, void* out, hipStream_t st) {
  const NormArgs a = args_of(s);
#define GDN_NORM_FWD(MODE)                                                                     \
  hipLaunchKernelGGL((norm_fwd_kernel<T, VEC, TPR, NC, MODE>), dim3((unsigned)blocks),         \
                     dim3(kBlock<TPR>), 0, st, (const T*)x, weight, bias, (const T*)z, (T*)out, a)
  if (!z)
    GDN_NORM_FWD(kModeNone);
  else if (s.gate_first)
    GDN_NORM_FWD(kModeFirst);
  else
    GDN_NORM_FWD(kModeLast);
#undef GDN_NORM_FWD
  return hipGetLastError();
}

template <typename T, int VEC, int TPR, int NC>
hipError_t bwd_k(const NormShape& s, int64_t blocks, const void* x, const float* weight,
                 const float* bias, const void* z, const void* dout, void* dx, void* dz,
                 float* partial, hipStream_t st) {
  const NormArgs a = args_of(s);
#define GDN_NORM_BWD(MODE)                                                                      \
  hipLaunchKernelGGL((norm_bwd_kernel<T, VEC, TPR, NC, MODE>), dim3((unsigned)blocks),          \
                     dim3(kBlock<TPR>), 0, st, (const T*)x, weight, bias, (const T*)z,          \
                     (const T*)dout, (T*)dx, (T*)dz, partial, a)
  if (!z)
    GDN_NORM_BWD(kModeNone);
  else if (s.gate_first)
    GDN_NORM_BWD(kModeFirst);
  else
    GDN_NORM_BWD(kModeLast);
#undef GDN_NORM_BWD
  return hipGetLastError();
}

#define GDN_NORM_PICK(F, ...)                                         \
  switch (p.tpr * 100 + p.nc) {                                       \
    case 801: return F<T, VEC, 8, 1>(__VA_ARGS__);                    \
    case 1601: return F<T, VEC, 16, 1>(__VA_ARGS__);                  \
    case 3201: return F<T, VEC, 32, 1>(__VA_ARGS__);                  \
    case 6401: return F<T, VEC, 64, 1>(__VA_ARGS__);                  \
    case 6402: return F<T, VEC, 64, 2>(__VA_ARGS__);                  \
    case 25601: return F<T, VEC, 256, 1>(__VA_ARGS__);                \
    case 25602: return F<T, VEC, 256, 2>(__VA_ARGS__);                \
    case 51202: return F<T, VEC, 512, 2>(__VA_ARGS__);                \
    case 102402: return F<T, VEC, 1024, 2>(__VA_ARGS__);              \
  }                                                                   \
  if constexpr (VEC < 8)                                              \
    if (p.tpr == 1024 && p.nc == 4)                                   \
      return F<T, VEC, 1024, 4>(__VA_ARGS__);                         \
  if constexpr (VEC == 1)                                             \
    if (p.tpr == 1024 && p.nc == 16)                                  \
      return F<T, VEC, 1024, 16>(__VA_ARGS__);                        \
  return hipErrorInvalidValue

template <typename T, int VEC>
hipError_t fwd_v(const NormShape& s, const Pick& p, const void* x, const float* weight,
                 const float* bias, const void* z, void* out, hipStream_t st) {
  GDN_NORM_PICK(fwd_k, s, fwd_blocks(s, p), x, weight, bias, z, out, st);
}

template <typename T, int VEC>
hipError_t bwd_v(const NormShape& s, const Pick& p, const void* x, const float* weight,
                 const float* bias, const void* z, const void* dout, void* dx, void* dz,
                 float* partial, hipStream_t st) {
  GDN_NORM_PICK(bwd_k, s, bwd_blocks(s, p), x, weight, bias, z, dout, dx, dz, partial, st);
}
#undef GDN_NORM_PICK

}  // namespace

hipError_t launch_norm_fwd(const NormShape& s, const void* x, const float* weight,
                           const float* bias, const void* z, void* out, hipStream_t st) {
  const Pick p = pick(s);
  if (s.bf16)
    return s.vec ? fwd_v<__bf16, 8>(s, p, x, weight, bias, z, out, st)
                 : fwd_v<__bf16, 1>(s, p, x, weight, bias, z, out, st);
  return s.vec ? fwd_v<float, 4>(s, p, x, weight, bias, z, out, st)
               : fwd_v<float, 1>(s, p, x, weight, bias, z, out, st);
}

size_t norm_bwd_workspace(const NormShape& s) {
  NormShape t = s;
  int64_t blocks = 0;
  for (const bool vec : {false, true}) {  // whichever of the two serves the call
    t.vec = vec;
    const int64_t b = bwd_blocks(t, pick(t));
    blocks = b > blocks ? b : blocks;
  }
  return align256((size_t)blocks * 2 * (size_t)s.dim * sizeof(float));
}

hipError_t launch_norm_bwd(const NormShape& s, const void* x, const float* weight,
                           const float* bias, const void* z, const void* dout, void* dx, void* dz,
                           float* dweight, float* dbias, float* ws, hipStream_t st) {
  const Pick p = pick(s);
  const int64_t blocks = bwd_blocks(s, p);
  if (blocks > 0) {
    hipError_t e;
    if (s.bf16)
      e = s.vec ? bwd_v<__bf16, 8>(s, p, x, weight, bias, z, dout, dx, dz, ws, st)
                : bwd_v<__bf16, 1>(s, p, x, weight, bias, z, dout, dx, dz, ws, st);
    else
      e = s.vec ? bwd_v<float, 4>(s, p, x, weight, bias, z, dout, dx, dz, ws, st)
                : bwd_v<float, 1>(s, p, x, weight, bias, z, dout, dx, dz, ws, st);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((unsigned)cdiv(s.dim, kSumCols), 2),
                     dim3(kSumCols * kSumRows), 0, st, ws, (int)blocks, s.dim, dweight, dbias);
  return hipGetLastError();
}

}  // namespace layer
}  // namespace gdn
