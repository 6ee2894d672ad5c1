// Low-rank adapters of a batch's requests beside a projection that they share:
//   out = base + scaling[a] (x A[a]^T) B[a]^T,   a the adapter of the row's request.
// A workgroup per row: the R sums over K by its waves in turn, then the M outputs.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void adapter_kernel(AdapterShape s, const T* x,
                                                           const T* base, const T* A, const T* B,
                                                           const float* scaling,
                                                           const int64_t* idx, const int64_t* cu,
                                                           T* out) {
  __shared__ float low[128];
  const int64_t t = blockIdx.x;
  if (cu && (t < cu[0] || t >= cu[s.B])) return;
  const int64_t a = idx[cu ? request_of(cu, s.B, t) : t];
  const bool some = a >= 0 && a < s.adapters;
  if (some) {
    for (int r = threadIdx.x >> 6; r < s.R; r += kThreads / 64) {
      const T* const w = A + (a * s.R + r) * s.K;
      float sum = 0.f;
      for (int k = threadIdx.x & 63; k < s.K; k += 64)
        sum = __builtin_fmaf((float)x[t * s.ldx + k], (float)w[k], sum);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off, 64);
      if ((threadIdx.x & 63) == 0) low[r] = scaling[a] * sum;
    }
  }
  __syncthreads();
  for (int m = threadIdx.x; m < s.M; m += kThreads) {
    float sum = 0.f;
    if (some)
      for (int r = 0; r < s.R; ++r)
        sum = __builtin_fmaf(low[r], (float)B[(a * s.M + m) * s.R + r], sum);
    out[t * s.ldout + m] = (T)((float)base[t * s.ldbase + m] + sum);
  }
}

template <typename T>
hipError_t launch(const AdapterShape& s, const void* x, const void* base, const void* A,
                  const void* B, const float* scaling, const int64_t* idx, const int64_t* cu,
                  void* out, hipStream_t st) {
  hipLaunchKernelGGL(adapter_kernel<T>, dim3((unsigned)s.N), dim3(kThreads), 0, st, s, (const T*)x,
                     (const T*)base, (const T*)A, (const T*)B, scaling, idx, cu, (T*)out);
  return hipGetLastError();
}

}  // namespace

size_t adapter_workspace(const AdapterShape&) { return 0; }

bool adapter_grids_fit(const AdapterShape& s) { return grid_ok(s.N, kThreads); }

hipError_t launch_adapter(const AdapterShape& s, const void* x, const void* base, const void* A,
                          const void* B, const float* scaling, const int64_t* idx,
                          const int64_t* cu, void* out, char*, hipStream_t st) {
  return s.bf16 ? launch<__bf16>(s, x, base, A, B, scaling, idx, cu, out, st)
                : launch<float>(s, x, base, A, B, scaling, idx, cu, out, st);
}

}  // namespace layer
}  // namespace gdn
