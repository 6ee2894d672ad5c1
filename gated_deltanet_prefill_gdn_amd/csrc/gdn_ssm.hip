// Selective state space scan token by token: one step for single tokens, and short requests of a
// prompt call, where a chunk of 64 rows would be mostly padding.
//
//   d = softplus(dt + dt_bias),  a = exp(-exp(A_log) d),  S <- a S + d x B^T,  out = S C + D x
//
// Row i of S (dv x dk, fp32) depends on x[i] alone, so rows are independent: a group of dk / 8
// lanes holds one row, 8 fp32 per lane, and a workgroup covers kRowsPerBlock rows of one
// (request, head). The state is read once, stays in registers over the request's tokens and is
// written once. With one token per request (decode) the kernel is bound by the state's bytes.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kTokenThreads = 256;
// Rows of a lane group. For one token two keep enough state loads in flight (512 requests, 32
// heads of 128 x 128: 369 us, 5.9 TB/s, with two, 400 with four, 565 with one); with several
// tokens four share each load of B and C (four tokens: 405 us, 460 with two).
template <int DK, bool ONE>
constexpr int kRows = ONE || DK == 64 ? 2 : 4;
template <int DK, bool ONE>
constexpr int kRowsPerBlock = (64 / (DK / 8)) * kRows<DK, ONE> * (kTokenThreads / 64);
static_assert(kRowsPerBlock<64, false> == 64 && kRowsPerBlock<128, false> == 64 &&
                  kRowsPerBlock<256, false> == 32 && kRowsPerBlock<64, true> == 64 &&
                  kRowsPerBlock<128, true> == 32 && kRowsPerBlock<256, true> == 16,
              "a workgroup's rows divide dv (64, 128 or 256)");

__device__ __forceinline__ float softplusf(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// x from another lane of the same 16-lane row, chosen by a DPP control code.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}

// Sum over an aligned group of LPR lanes, left in every lane of it.
template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
  static_assert(LPR == 8 || LPR == 16 || LPR == 32, "8 to 32 lanes per row");
  x += dpp<0xB1>(x);   // lane ^ 1
  x += dpp<0x4E>(x);   // lane ^ 2
  x += dpp<0x141>(x);  // the other quad of the half-row, mirrored
  if constexpr (LPR >= 16) x += dpp<0x140>(x);  // the other half of the row, mirrored
  if constexpr (LPR >= 32) x += __shfl_xor(x, 16, 64);
  return x;
}

// This lane's eight entries of a row of DK: 4 gl .. and DK / 2 + 4 gl .., so that a wave's load
// covers contiguous half rows.
template <int DK>
__device__ __forceinline__ void load8(const float* row, int gl, float (&x)[8]) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(row + 4 * gl);
  const f32x4 hi = *reinterpret_cast<const f32x4*>(row + DK / 2 + 4 * gl);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lo[i];
    x[4 + i] = hi[i];
  }
}
template <int DK>
__device__ __forceinline__ void load8(const __bf16* row, int gl, float (&x)[8]) {
  const bf16x4 lo = *reinterpret_cast<const bf16x4*>(row + 4 * gl);
  const bf16x4 hi = *reinterpret_cast<const bf16x4*>(row + DK / 2 + 4 * gl);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = (float)lo[i];
    x[4 + i] = (float)hi[i];
  }
}

// ONE: one token per request, row b (cu is not read).
template <int DK, typename T, bool ONE>
__global__ __launch_bounds__(kTokenThreads) void ssm_token_kernel(
    const T* __restrict__ cm, const T* __restrict__ bm, const T* __restrict__ x,
    const float* __restrict__ dt, const float* __restrict__ A_log,
    const float* __restrict__ dt_bias, const float* __restrict__ D,
    float* __restrict__ state_pool, const int64_t* __restrict__ idx,
    const int64_t* __restrict__ cu, T* __restrict__ out, int64_t N, int64_t pool, int H, int HV,
    int DV, int nrb, int64_t max_len) {
  constexpr int LPR = DK / 8, RPW = 64 / LPR, NR = kRows<DK, ONE>, RWV = RPW * NR;
  const uint32_t pair = blockIdx.x / (uint32_t)nrb;
  const int rb = (int)(blockIdx.x - pair * (uint32_t)nrb);
  const uint32_t b = pair / (uint32_t)HV;
  const int hv = (int)(pair - b * (uint32_t)HV), h = hv / (HV / H);
  int64_t t = b, t_end = (int64_t)b + 1;
  if constexpr (!ONE) {
    t = cu[b] < 0 ? 0 : cu[b];
    t_end = cu[b + 1] < N ? cu[b + 1] : N;
  }
  const int64_t slot = idx[b];
  if (t >= t_end || t_end - t > max_len || slot < 0 || slot >= pool) return;
  const int l = threadIdx.x & 63, gl = l % LPR;
  const int r0 = rb * kRowsPerBlock<DK, ONE> + (threadIdx.x >> 6) * RWV + l / LPR;
  float* const sp = state_pool + ((slot * HV + hv) * (int64_t)DV + r0) * DK + 4 * gl;
  f32x4 s[NR][2];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    s[j][0] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(sp + j * RPW * DK));
    s[j][1] =
        __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(sp + j * RPW * DK + DK / 2));
  }
  const float rate = expf(A_log[hv]), dtb = dt_bias[hv], dd = D ? D[hv] : 0.f;
  const float decay = rate > 3e38f ? 3e38f : rate;  // finite, so that no step means no decay
  for (; t < t_end; ++t) {
    const int64_t th = t * HV + hv;
    float bb[8], cc[8], xr[NR];
    load8<DK>(bm + (t * H + h) * DK, gl, bb);
    load8<DK>(cm + (t * H + h) * DK, gl, cc);
#pragma unroll
    for (int j = 0; j < NR; ++j) xr[j] = (float)x[th * DV + r0 + j * RPW];
    const float step = softplusf(dt[th] + dtb), a = expf(-decay * step);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const float u = step * xr[j];
      float o = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float se = __builtin_fmaf(a, s[j][e / 4][e % 4], u * bb[e]);
        s[j][e / 4][e % 4] = se;
        o = __builtin_fmaf(se, cc[e], o);
      }
      o = group_sum<LPR>(o);
      if (gl == 0) out[th * DV + r0 + j * RPW] = (T)__builtin_fmaf(dd, xr[j], o);
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    __builtin_nontemporal_store(s[j][0], reinterpret_cast<f32x4*>(sp + j * RPW * DK));
    __builtin_nontemporal_store(s[j][1], reinterpret_cast<f32x4*>(sp + j * RPW * DK + DK / 2));
  }
}

int rows_per_block(int dk, bool one) {
  return dk == 256 ? (one ? kRowsPerBlock<256, true> : kRowsPerBlock<256, false>)
         : dk == 128 ? (one ? kRowsPerBlock<128, true> : kRowsPerBlock<128, false>)
                     : kRowsPerBlock<64, true>;
}

int64_t token_blocks(const SsmShape& s, bool one) {
  return s.B * s.HV * (s.dv / rows_per_block(s.dk, one));
}

template <int DK, typename T, bool ONE>
hipError_t launch_token(const SsmShape& s, const void* C, const void* B, const void* x,
                        const float* dt, const float* A_log, const float* dt_bias, const float* D,
                        float* state, const int64_t* idx, const int64_t* cu, void* out,
                        int64_t max_len, hipStream_t st) {
  hipLaunchKernelGGL((ssm_token_kernel<DK, T, ONE>), dim3((unsigned)token_blocks(s, ONE)),
                     dim3(kTokenThreads), 0, st, (const T*)C, (const T*)B, (const T*)x, dt, A_log,
                     dt_bias, D, state, idx, cu, (T*)out, s.N, s.pool, s.H, s.HV, s.dv,
                     s.dv / kRowsPerBlock<DK, ONE>, max_len);
  return hipGetLastError();
}

template <bool ONE>
hipError_t launch_token_any(const SsmShape& s, const void* C, const void* B, const void* x,
                            const float* dt, const float* A_log, const float* dt_bias,
                            const float* D, float* state, const int64_t* idx, const int64_t* cu,
                            void* out, int64_t max_len, hipStream_t st) {
#define GDN_SSM_CASE(DK)                                                                     \
  if (s.dk == DK)                                                                            \
    return s.bf16 ? launch_token<DK, __bf16, ONE>(s, C, B, x, dt, A_log, dt_bias, D, state,  \
                                                  idx, cu, out, max_len, st)                 \
                  : launch_token<DK, float, ONE>(s, C, B, x, dt, A_log, dt_bias, D, state,   \
                                                 idx, cu, out, max_len, st);
  GDN_SSM_CASE(64)
  GDN_SSM_CASE(128)
  GDN_SSM_CASE(256)
#undef GDN_SSM_CASE
  return hipErrorInvalidValue;
}

}  // namespace

bool ssm_token_grid_fits(const SsmShape& s) {
  return grid_ok(token_blocks(s, true), kTokenThreads);  // the larger of the two grids
}

hipError_t launch_ssm_decode(const SsmShape& s, const void* C, const void* B, const void* x,
                             const float* dt, const float* A_log, const float* dt_bias,
                             const float* D, float* state, const int64_t* idx, void* out,
                             hipStream_t st) {
  return launch_token_any<true>(s, C, B, x, dt, A_log, dt_bias, D, state, idx, nullptr, out, 1, st);
}

hipError_t launch_ssm_short(const SsmShape& s, const void* C, const void* B, const void* x,
                            const float* dt, const float* A_log, const float* dt_bias,
                            const float* D, float* state, const int64_t* idx, const int64_t* cu,
                            void* out, int64_t max_len, hipStream_t st) {
  return launch_token_any<false>(s, C, B, x, dt, A_log, dt_bias, D, state, idx, cu, out, max_len,
                                 st);
}

}  // namespace layer
}  // namespace gdn
