// Linear attention token by token: one step for single tokens, and short requests of a prompt call,
// where a chunk of 64 rows would be mostly padding.
//
//   S <- a S + v k^T,  out = c S q,   a = e^{log_decay}
//
// Row i of S (dv x dk, fp32) depends on v[i] alone, so rows are independent: a group of dk / 8
// lanes holds one row, 8 fp32 per lane, and a workgroup covers kRowsPerBlock rows of one
// (request, head). The state is read once, stays in registers over the request's tokens and is
// written once. With one token per request (decode) the kernel is bound by the state's bytes: 512
// requests, 32 heads of 128 x 128, bf16: 2.17 GB in 371 us, 5.8 TB/s (a copy of 1 GiB reaches 5.2
// here); 16 heads of one request 3.2 us, a launch's latency.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kTokenThreads = 256;
// Rows of a lane group: for one token two keep enough state loads in flight, with several tokens
// four share each load of q and k.
template <int DK, bool ONE>
constexpr int kRows = ONE || DK == 64 ? 2 : 4;
template <int DK, bool ONE>
constexpr int kRowsPerBlock = (64 / (DK / 8)) * kRows<DK, ONE> * (kTokenThreads / 64);
static_assert(kRowsPerBlock<64, false> == 64 && kRowsPerBlock<128, false> == 64 &&
                  kRowsPerBlock<256, false> == 32 && kRowsPerBlock<64, true> == 64 &&
                  kRowsPerBlock<128, true> == 32 && kRowsPerBlock<256, true> == 16,
              "a workgroup's rows divide dv (64, 128 or 256)");

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
template <int DK, typename T>
__device__ __forceinline__ void load8(const T* row, int gl, float (&x)[8]) {
  float lo[4], hi[4];
  load_vec<4>(row + 4 * gl, lo);
  load_vec<4>(row + DK / 2 + 4 * gl, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lo[i];
    x[4 + i] = hi[i];
  }
}

// ONE: one token per request, row b (cu is not read).
template <int DK, typename T, bool ONE>
__global__ __launch_bounds__(kTokenThreads) void linear_token_kernel(
    LinearShape s, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ log_decay, float* __restrict__ state_pool,
    const int64_t* __restrict__ idx, const int64_t* __restrict__ cu, T* __restrict__ out, int nrb,
    int64_t max_len) {
  constexpr int LPR = DK / 8, RPW = 64 / LPR, NR = kRows<DK, ONE>, RWV = RPW * NR;
  const uint32_t pair = blockIdx.x / (uint32_t)nrb;
  const int rb = (int)(blockIdx.x - pair * (uint32_t)nrb);
  const uint32_t b = pair / (uint32_t)s.HV;
  const int hv = (int)(pair - b * (uint32_t)s.HV), h = hv / (s.HV / s.H);
  int64_t t = b, t_end = (int64_t)b + 1;
  if constexpr (!ONE) {
    t = cu[b] < 0 ? 0 : cu[b];
    t_end = cu[b + 1] < s.N ? cu[b + 1] : s.N;
  }
  const int64_t slot = state_pool ? idx[b] : 0;
  if (t >= t_end || t_end - t > max_len || (state_pool && (slot < 0 || slot >= s.pool))) return;
  const int l = threadIdx.x & 63, gl = l % LPR;
  const int r0 = rb * kRowsPerBlock<DK, ONE> + (threadIdx.x >> 6) * RWV + l / LPR;
  float* const sp = state_pool + ((slot * s.HV + hv) * (int64_t)s.dv + r0) * DK + 4 * gl;
  f32x4 st[NR][2];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int half = 0; half < 2; ++half)
      st[j][half] = ONE || state_pool
                        ? __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(
                              sp + j * RPW * DK + half * (DK / 2)))
                        : f32x4{0.f, 0.f, 0.f, 0.f};
  const float g = log_decay[hv], a = g > 0.f ? 1.f : expf(g);
  for (; t < t_end; ++t) {
    float kk[8], qq[8], vr[NR];
    load8<DK>(k + t * s.ldk + h * DK, gl, kk);
    load8<DK>(q + t * s.ldq + h * DK, gl, qq);
#pragma unroll
    for (int j = 0; j < NR; ++j)
      vr[j] = (float)v[t * s.ldv + (int64_t)hv * s.dv + r0 + j * RPW];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      float o = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float se = __builtin_fmaf(a, st[j][e / 4][e % 4], vr[j] * kk[e]);
        st[j][e / 4][e % 4] = se;
        o = __builtin_fmaf(se, qq[e], o);
      }
      o = group_sum<LPR>(o);
      if (gl == 0) out[(t * s.HV + hv) * s.dv + r0 + j * RPW] = (T)(s.scale * o);
    }
  }
  if (!ONE && !state_pool) return;
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int half = 0; half < 2; ++half)
      __builtin_nontemporal_store(
          st[j][half], reinterpret_cast<f32x4*>(sp + j * RPW * DK + half * (DK / 2)));
}

int rows_per_block(int dk, bool one) {
  return dk == 256 ? (one ? kRowsPerBlock<256, true> : kRowsPerBlock<256, false>)
         : dk == 128 ? (one ? kRowsPerBlock<128, true> : kRowsPerBlock<128, false>)
                     : kRowsPerBlock<64, true>;
}

int64_t token_blocks(const LinearShape& s, bool one) {
  return s.B * s.HV * (s.dv / rows_per_block(s.dk, one));
}

template <bool ONE>
hipError_t launch_token(const LinearShape& s, const void* q, const void* k, const void* v,
                        const float* log_decay, float* state, const int64_t* idx,
                        const int64_t* cu, void* out, int64_t max_len, hipStream_t st) {
  const dim3 grid((unsigned)token_blocks(s, ONE)), threads(kTokenThreads);
  const int nrb = s.dv / rows_per_block(s.dk, ONE);
#define GDN_LINEAR_CASE(DK, T)                                                                  \
  if (s.dk == DK && s.bf16 == (sizeof(T) == 2)) {                                               \
    hipLaunchKernelGGL((linear_token_kernel<DK, T, ONE>), grid, threads, 0, st, s, (const T*)q, \
                       (const T*)k, (const T*)v, log_decay, state, idx, cu, (T*)out, nrb,       \
                       max_len);                                                                \
    return hipGetLastError();                                                                   \
  }
  GDN_LINEAR_CASE(64, __bf16)
  GDN_LINEAR_CASE(128, __bf16)
  GDN_LINEAR_CASE(256, __bf16)
  GDN_LINEAR_CASE(64, float)
  GDN_LINEAR_CASE(128, float)
  GDN_LINEAR_CASE(256, float)
#undef GDN_LINEAR_CASE
  return hipErrorInvalidValue;
}

}  // namespace

bool linear_token_grid_fits(const LinearShape& s) {
  return grid_ok(token_blocks(s, true), kTokenThreads);  // the larger of the two grids
}

hipError_t launch_linear_decode(const LinearShape& s, const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, const int64_t* idx,
                                void* out, hipStream_t st) {
  return launch_token<true>(s, q, k, v, log_decay, state, idx, nullptr, out, 1, st);
}

hipError_t launch_linear_short(const LinearShape& s, const void* q, const void* k, const void* v,
                               const float* log_decay, float* state, const int64_t* idx,
                               const int64_t* cu, void* out, int64_t max_len, hipStream_t st) {
  return launch_token<false>(s, q, k, v, log_decay, state, idx, cu, out, max_len, st);
}

}  // namespace layer
}  // namespace gdn
