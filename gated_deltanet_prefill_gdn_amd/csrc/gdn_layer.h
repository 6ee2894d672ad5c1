// Internal declarations of the layer operators around the recurrence: short causal
// convolution, selective state space scan, gated norm. Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {
namespace layer {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Elements of one 16-byte vector.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// VEC consecutive elements at p, as fp32. VEC > 1 needs p aligned to VEC elements (at most 16
// bytes are loaded at a time).
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      const f32x4 v = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * i + e] = v[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = p[i];
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __bf16* p, float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
  } else if constexpr (VEC == 4) {
    const bf16x4 v = *reinterpret_cast<const bf16x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)v[e];
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) x[i] = (float)p[i];
  }
}

// The same in the stored type: what a load leaves in registers until its use (half the registers
// of fp32 for bf16).
template <typename T, int VEC>
struct Raw {
  typedef T vec_t __attribute__((ext_vector_type(VEC)));
  vec_t v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const vec_t*>(p); }
  __device__ __forceinline__ void zero() { v = (vec_t)(T)0.f; }
  __device__ __forceinline__ float operator[](int e) const { return (float)v[e]; }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = (T)0.f; }
  __device__ __forceinline__ float operator[](int) const { return (float)v; }
};

// Rounded once to the stored type (round to nearest even, NaN stays NaN).
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i)
      reinterpret_cast<f32x4*>(p)[i] = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = x[i];
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__bf16* p, const float (&x)[VEC]) {
  if constexpr (VEC == 8) {
    bf16x8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (__bf16)x[e];
    *reinterpret_cast<bf16x8*>(p) = v;
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<bf16x4*>(p) =
        bf16x4{(__bf16)x[0], (__bf16)x[1], (__bf16)x[2], (__bf16)x[3]};
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) p[i] = (__bf16)x[i];
  }
}

// 1 / (1 + e^-x): e^-x overflows to infinity only where the quotient is below 2^-126.
__device__ __forceinline__ float sigmoidf(float x) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-x));
}

// Request that owns token t: cu[b] <= t < cu[b + 1], by bisection; t < cu[B] and cu[0] <= t.
__device__ __forceinline__ int64_t request_of(const int64_t* __restrict__ cu, int64_t B,
                                              int64_t t) {
  int64_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A launch of `blocks` workgroups of `threads` work-items along x: the dispatch packet holds
// the grid size in work-items as 32 bits.
inline bool grid_ok(int64_t blocks, int threads) {
  return blocks >= 0 && blocks <= 0x7FFFFFFF && blocks * (int64_t)threads <= (int64_t)0xFFFFFFFF;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// ---- short causal convolution
struct ConvShape {
  int64_t N, B, pool, x_stride, dx_stride;
  int ch, c1, c2;  // all channels; first channel of out1 and of out2
  int W;
  bool bf16, dout_bf16, silu, vec;  // vec: 16-byte vectors everywhere
};
hipError_t launch_conv_fwd(const ConvShape& s, const void* x, const float* weight,
                           const float* bias, void* state, const int64_t* idx, const int64_t* cu,
                           void* const out[3], hipStream_t st);
hipError_t launch_conv_decode(const ConvShape& s, const void* x, const float* weight,
                              const float* bias, void* state, const int64_t* idx,
                              void* const out[3], hipStream_t st);
size_t conv_bwd_workspace(const ConvShape& s);
hipError_t launch_conv_bwd(const ConvShape& s, const void* x, const float* weight,
                           const float* bias, const void* state, const int64_t* idx,
                           const int64_t* cu, const void* const dout[3], const float* dstate,
                           void* dx, float* dweight, float* dbias, float* dstate0, float* ws,
                           hipStream_t st);
bool conv_grids_fit(const ConvShape& s, bool backward);

// ---- gated norm
struct NormShape {
  int64_t N, x_stride, z_stride, dz_stride;
  int heads, dim;
  bool bf16, rms, gate_first, vec;
  float eps;
};
hipError_t launch_norm_fwd(const NormShape& s, const void* x, const float* weight,
                           const float* bias, const void* z, void* out, hipStream_t st);
size_t norm_bwd_workspace(const NormShape& s);
hipError_t launch_norm_bwd(const NormShape& s, const void* x, const float* weight,
                           const float* bias, const void* z, const void* dout, void* dx, void* dz,
                           float* dweight, float* dbias, float* ws, hipStream_t st);

// ---- selective state space scan
struct SsmShape {
  int64_t N, B, pool;
  int H, HV, dk, dv;
  bool bf16;
};
size_t ssm_workspace(const SsmShape& s);
bool ssm_prefill_grids_fit(const SsmShape& s);
bool ssm_token_grid_fits(const SsmShape& s);
hipError_t launch_ssm_prefill(const SsmShape& s, const void* C, const void* B, const void* x,
                              const float* dt, const float* A_log, const float* dt_bias,
                              const float* D, float* state, const int64_t* idx,
                              const int64_t* cu, void* out, char* ws, hipStream_t st);
hipError_t launch_ssm_decode(const SsmShape& s, const void* C, const void* B, const void* x,
                             const float* dt, const float* A_log, const float* dt_bias,
                             const float* D, float* state, const int64_t* idx, void* out,
                             hipStream_t st);

// Requests of at most max_len tokens, token by token; the others are left alone.
hipError_t launch_ssm_short(const SsmShape& s, const void* C, const void* B, const void* x,
                            const float* dt, const float* A_log, const float* dt_bias,
                            const float* D, float* state, const int64_t* idx, const int64_t* cu,
                            void* out, int64_t max_len, hipStream_t st);

}  // namespace layer
}  // namespace gdn
