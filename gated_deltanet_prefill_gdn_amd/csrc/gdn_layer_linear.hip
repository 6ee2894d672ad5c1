// Linear attention with a fixed decay for each head, token by token.
//
// Every call is made of walks of one recurrence over the tokens of a request,
//   W <- a W + w v k^T,   out = r W q,   a = e^{log_decay},
// W (rows x DK, fp32) with the row of v: the forward call walks (q, k, v) over S; the gradients are
// dq: (dout, v, k) over S^T, and from the last token to the first dv: (k, q, dout) over D and
// dk: (v, dout, q) over D^T, D the gradient of the state. Row i of W depends on v[i] alone, so rows
// are independent: a group of DK / 8 lanes holds one row, 8 fp32 per lane.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kTokenThreads = 256;

struct Walk {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;  // elements between tokens
  int rq, rk, rv;         // value heads per head of q, k and v
  void* out;              // [N, HV, rows] dense
  const float* first;     // states in front of the walk, or NULL for zero
  float* last;            // ... behind it, or NULL
  bool first_pool, last_pool;  // by slot of the pool, else by request
  int64_t row_step, col_step;  // of a state's entries
  float read, write;
  bool back;  // from the last token to the first; the decay comes behind a token
};

struct WalkArgs {
  const float* log_decay;
  const int64_t *idx, *cu;
  int64_t N, npool;
  int HV, rows;
};

__device__ __forceinline__ float decay_of(float g) {  // (NaN stays NaN)
  return g > 0.f ? 1.f : expf(g);
}

template <int DK, typename T, typename TO>
__global__ __launch_bounds__(kTokenThreads) void linear_walk_kernel(Walk w, WalkArgs a) {
  constexpr int LPR = DK / 8, PER = kTokenThreads / LPR;
  const int nrb = a.rows / PER;
  const int64_t pair = blockIdx.x / (unsigned)nrb;
  const int row = (int)(blockIdx.x - pair * nrb) * PER + threadIdx.x / LPR, gl = threadIdx.x % LPR;
  const int64_t b = pair / a.HV;
  const int hv = (int)(pair - b * a.HV);
  int64_t t0 = b, t1 = b + 1;
  if (a.cu) {
    t0 = a.cu[b] < 0 ? 0 : a.cu[b];
    t1 = a.cu[b + 1] < a.N ? a.cu[b + 1] : a.N;
  }
  const int64_t slot = a.idx ? a.idx[b] : b;
  const bool live = !a.idx || (slot >= 0 && slot < a.npool);
  const int64_t plane = (int64_t)a.rows * DK;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  if (w.first && live) {
    const float* p = w.first + ((w.first_pool ? slot : b) * a.HV + hv) * plane + row * w.row_step;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = p[(8 * gl + e) * w.col_step];
  }
  const float decay = decay_of(a.log_decay[hv]);
  const int64_t n = live && t1 > t0 ? t1 - t0 : 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t t = w.back ? t1 - 1 - i : t0 + i;
    const T* const q = reinterpret_cast<const T*>(w.q) + t * w.ldq + (hv / w.rq) * DK + 8 * gl;
    const T* const k = reinterpret_cast<const T*>(w.k) + t * w.ldk + (hv / w.rk) * DK + 8 * gl;
    const float v =
        w.write * (float)reinterpret_cast<const T*>(w.v)[t * w.ldv + (int64_t)(hv / w.rv) * a.rows + row];
    const float before = w.back ? 1.f : decay;
    float o = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] = __builtin_fmaf(before, s[e], v * (float)k[e]);
      o = __builtin_fmaf(s[e], (float)q[e], o);
    }
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) o += __shfl_xor(o, off, 64);
    if (gl == 0) reinterpret_cast<TO*>(w.out)[(t * a.HV + hv) * a.rows + row] = (TO)(w.read * o);
    if (w.back)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] *= decay;
  }
  if (w.last && (live || !w.last_pool)) {
    float* p = w.last + ((w.last_pool ? slot : b) * a.HV + hv) * plane + row * w.row_step;
#pragma unroll
    for (int e = 0; e < 8; ++e) p[(8 * gl + e) * w.col_step] = s[e];
  }
}

// dq and dk of a group's head: the sum over its value heads, in order.
template <typename T>
__global__ __launch_bounds__(256) void linear_group_sum_kernel(const float* part, T* out,
                                                               const int64_t* idx,
                                                               const int64_t* cu, int64_t B,
                                                               int64_t N, int64_t npool, int H,
                                                               int rep, int d) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N * H * d) return;
  const int64_t t = i / ((int64_t)H * d);
  if (t < cu[0] || t >= cu[B]) return;
  if (idx) {
    const int64_t slot = idx[request_of(cu, B, t)];
    if (slot < 0 || slot >= npool) return;
  }
  const int64_t th = i / d;
  float s = 0.f;
  for (int r = 0; r < rep; ++r) s += part[(th * rep + r) * d + (i - th * d)];
  out[i] = (T)s;
}

template <typename T, typename TO>
hipError_t launch_walk(const Walk& w, const WalkArgs& a, int64_t B, int DK, hipStream_t st) {
  const int64_t blocks = B * a.HV * (a.rows / (kTokenThreads / (DK / 8)));
  const auto kernel = DK == 64    ? linear_walk_kernel<64, T, TO>
                      : DK == 128 ? linear_walk_kernel<128, T, TO>
                                  : linear_walk_kernel<256, T, TO>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kTokenThreads), 0, st, w, a);
  return hipGetLastError();
}

template <typename T>
hipError_t forward(const LinearShape& s, const void* q, const void* k, const void* v,
                   const float* log_decay, float* state, const int64_t* idx, const int64_t* cu,
                   void* out, hipStream_t st) {
  const int rep = s.HV / s.H;
  const Walk w{q, k, v, s.ldq, s.ldk, s.ldv, rep, rep, 1, out, state, state, true, true,
               s.dk, 1, s.scale, 1.f, false};
  const WalkArgs a{log_decay, state ? idx : nullptr, cu, s.N, s.pool, s.HV, s.dv};
  return launch_walk<T, T>(w, a, s.B, s.dk, st);
}

template <typename T>
hipError_t backward(const LinearShape& s, const void* q, const void* k, const void* v,
                    const float* log_decay, const float* state, const int64_t* idx,
                    const int64_t* cu, const void* dout, const float* dstate, void* dq, void* dk,
                    void* dv, float* dstate0, float* ws, hipStream_t st) {
  const int rep = s.HV / s.H;
  const int64_t ldo = (int64_t)s.HV * s.dv, part = s.N * s.HV * s.dk;
  const WalkArgs ak{log_decay, state ? idx : nullptr, cu, s.N, s.pool, s.HV, s.dk};
  const WalkArgs av{log_decay, state ? idx : nullptr, cu, s.N, s.pool, s.HV, s.dv};
  const Walk wq{dout, v, k, ldo, s.ldv, s.ldk, 1, 1, rep, rep > 1 ? ws : dq, state, nullptr, true,
                false, 1, s.dk, s.scale, 1.f, false};
  const Walk wk{v, dout, q, s.ldv, ldo, s.ldq, 1, 1, rep, rep > 1 ? ws + part : dk, dstate,
                nullptr, false, false, 1, s.dk, 1.f, s.scale, true};
  const Walk wv{k, q, dout, s.ldk, s.ldq, ldo, rep, rep, 1, dv, dstate, dstate0, false, false,
                s.dk, 1, 1.f, s.scale, true};
  hipError_t e;
  if (rep == 1) {
    if ((e = launch_walk<T, T>(wq, ak, s.B, s.dv, st)) != hipSuccess) return e;
    if ((e = launch_walk<T, T>(wk, ak, s.B, s.dv, st)) != hipSuccess) return e;
    return launch_walk<T, T>(wv, av, s.B, s.dk, st);
  }
  if ((e = launch_walk<T, float>(wq, ak, s.B, s.dv, st)) != hipSuccess) return e;
  if ((e = launch_walk<T, float>(wk, ak, s.B, s.dv, st)) != hipSuccess) return e;
  if ((e = launch_walk<T, T>(wv, av, s.B, s.dk, st)) != hipSuccess) return e;
  const int64_t n = s.N * s.H * s.dk;
  if (n == 0) return hipSuccess;
  for (int i = 0; i < 2; ++i) {
    hipLaunchKernelGGL(linear_group_sum_kernel<T>, dim3((unsigned)cdiv(n, 256)), dim3(256), 0, st,
                       ws + i * part, (T*)(i ? dk : dq), state ? idx : nullptr, cu, s.B, s.N,
                       s.pool, s.H, rep, s.dk);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

bool walk_grid_fits(const LinearShape& s, int DK, int rows) {
  return grid_ok(s.B * s.HV * (rows / (kTokenThreads / (DK / 8))), kTokenThreads);
}

}  // namespace

size_t linear_workspace(const LinearShape&) { return 0; }
size_t linear_bwd_workspace(const LinearShape& s) {
  return s.HV > s.H ? align256(2 * sizeof(float) * s.N * s.HV * s.dk) : 0;
}
bool linear_prefill_grids_fit(const LinearShape& s) { return walk_grid_fits(s, s.dk, s.dv); }
bool linear_decode_grid_fits(const LinearShape& s) { return walk_grid_fits(s, s.dk, s.dv); }
bool linear_bwd_grids_fit(const LinearShape& s) {
  return walk_grid_fits(s, s.dk, s.dv) && walk_grid_fits(s, s.dv, s.dk) &&
         grid_ok(cdiv(s.N * s.H * s.dk, 256), 256);
}

hipError_t launch_linear_prefill(const LinearShape& s, const void* q, const void* k, const void* v,
                                 const float* log_decay, float* state, const int64_t* idx,
                                 const int64_t* cu, void* out, char*, hipStream_t st) {
  return s.bf16 ? forward<__bf16>(s, q, k, v, log_decay, state, idx, cu, out, st)
                : forward<float>(s, q, k, v, log_decay, state, idx, cu, out, st);
}

hipError_t launch_linear_decode(const LinearShape& s, const void* q, const void* k, const void* v,
                                const float* log_decay, float* state, const int64_t* idx,
                                void* out, hipStream_t st) {
  return launch_linear_prefill(s, q, k, v, log_decay, state, idx, nullptr, out, nullptr, st);
}

hipError_t launch_linear_bwd(const LinearShape& s, const void* q, const void* k, const void* v,
                             const float* log_decay, const float* state, const int64_t* idx,
                             const int64_t* cu, const void* dout, const float* dstate, void* dq,
                             void* dk, void* dv, float* dstate0, char* ws, hipStream_t st) {
  return s.bf16 ? backward<__bf16>(s, q, k, v, log_decay, state, idx, cu, dout, dstate, dq, dk, dv,
                                   dstate0, (float*)ws, st)
                : backward<float>(s, q, k, v, log_decay, state, idx, cu, dout, dstate, dq, dk, dv,
                                  dstate0, (float*)ws, st);
}

}  // namespace layer
}  // namespace gdn
