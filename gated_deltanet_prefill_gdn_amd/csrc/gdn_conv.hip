// Short causal convolution over packed requests, its single-token form and its gradients.
//
// With u = a request's W - 1 history rows followed by its tokens, channel by channel:
//   pre[p] = bias + sum_{j < W} w[j] u[p + j],  out = silu(pre) or pre,  state <- last W - 1 of u.
// Gradients, with g = dout * silu'(pre), silu'(y) = s (1 + y (1 - s)), s = sigmoid(y):
//   dw[j] = sum_p g[p] u[p + j],  db = sum_p g[p],
//   du[e] = sum_{s < W} w[W - 1 - s] g[e + s]   (token e; g = 0 outside the request's tokens)
// plus the gradient of the final state for its rows.
//
// All three are bound by HBM: one pass over the token rows, a thread owning VEC channels (one
// 16-byte vector) and a run of tokens whose window slides through registers, so every input row
// is read once but for the W - 1 rows where runs meet. Measured, bf16, W = 4: 33860 tokens of 8192
// channels 220 us (5.2 TB/s), 512 single tokens of 8192 channels 12.3 us (5.6 TB/s), gradients of
// 16384 tokens of 6144 channels 167 us (5.0 TB/s) and 11 for the sums and the states' gradients.
#include "gdn_layer.h"

namespace gdn {
namespace layer {
namespace {

constexpr int kThreads = 256;

struct Outs {
  void* p[3];
  int c1, c2, ch;  // first channel of outputs 1 and 2, all channels
};

// Row base and row length of the output that channel c goes to (a vector never straddles two
// outputs: the vector path needs every channel count to be a multiple of VEC).
template <typename T>
__device__ __forceinline__ T* out_place(const Outs& o, int c, int64_t& ld) {
  if (c < o.c1) {
    ld = o.c1;
    return reinterpret_cast<T*>(o.p[0]) + c;
  }
  if (c < o.c2) {
    ld = o.c2 - o.c1;
    return reinterpret_cast<T*>(o.p[1]) + (c - o.c1);
  }
  ld = o.ch - o.c2;
  return reinterpret_cast<T*>(o.p[2]) + (c - o.c2);
}

template <int VEC, int W>
__device__ __forceinline__ void load_weights(const float* __restrict__ weight,
                                             const float* __restrict__ bias, int c,
                                             float (&w)[W][VEC], float (&b)[VEC]) {
  float t[VEC * W];  // rows c .. c + VEC - 1 of [CH, W] are contiguous
  if constexpr (VEC > 1) {
    load_vec<VEC * W>(weight + (int64_t)c * W, t);
  } else {  // only aligned to one weight
#pragma unroll
    for (int j = 0; j < W; ++j) t[j] = weight[(int64_t)c * W + j];
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[j][e] = t[e * W + j];
  if (bias) {
    load_vec<VEC>(bias + c, b);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) b[e] = 0.f;
  }
}

// The request under a thread's cursor. Tokens are clamped to [0, N), so a cu_seqlens that
// breaks its precondition cannot lead outside the arrays.
struct Cursor {
  int64_t req = 0, begin = 0, end = 0, slot = -1;
  bool live = false;  // false: a padding request, skipped
};
__device__ __forceinline__ void seek(Cursor& q, const int64_t* __restrict__ cu,
                                     const int64_t* __restrict__ idx, int64_t req, int64_t N,
                                     int64_t pool, bool stateful) {
  q.req = req;
  q.begin = cu[req] < 0 ? 0 : cu[req];
  q.end = cu[req + 1] > N ? N : cu[req + 1];
  q.slot = stateful ? idx[req] : 0;
  q.live = !stateful || (q.slot >= 0 && q.slot < pool);
}

// Row at position p of request q (p < 0: history row W - 1 + p, zero without a state pool).
template <typename T, int VEC, int W>
__device__ __forceinline__ void load_row(const T* __restrict__ x, int64_t x_stride,
                                         const T* state, int ch, int c, const Cursor& q,
                                         int64_t p, float (&r)[VEC]) {
  if (p >= 0) {
    load_vec<VEC>(x + (q.begin + p) * x_stride + c, r);
  } else if (state) {
    load_vec<VEC>(state + (q.slot * (W - 1) + (W - 1) + p) * (int64_t)ch + c, r);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) r[e] = 0.f;
  }
}

// A tile [t0, t0 + tile) of the token axis gives up the first W - 2 tokens after a request's
// first one to the tile that holds the first: that thread alone reads the request's history,
// and it writes the new state (from x, and from the history it holds) after reading it, so the
// pool is updated in place without a second launch.
template <int W>
__device__ __forceinline__ int64_t owned_from(int64_t t, const Cursor& q) {
  const int64_t pos = t - q.begin;
  if (pos == 0 || pos >= W - 1) return t;
  const int64_t to = q.begin + (W - 1);
  return to < q.end ? to : q.end;
}

template <typename T, int VEC, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(
    const T* __restrict__ x, int64_t x_stride, const float* __restrict__ weight,
    const float* __restrict__ bias, T* state, const int64_t* __restrict__ idx,
    const int64_t* __restrict__ cu, Outs outs, int64_t N, int64_t B, int64_t pool, int tile) {
  const int ch = outs.ch;
  const int c = (int)(blockIdx.y * kThreads + threadIdx.x) * VEC;
  if (c >= ch) return;
  const int64_t last = cu[B] < N ? cu[B] : N;  // rows behind the last request are padding
  int64_t t = (int64_t)blockIdx.x * tile;
  if (t < cu[0]) t = cu[0];
  int64_t stop = ((int64_t)blockIdx.x + 1) * tile;
  if (stop > last) stop = last;
  if (t >= stop) return;

  Cursor q;
  seek(q, cu, idx, request_of(cu, B, t), N, pool, state != nullptr);
  t = owned_from<W>(t, q);
  if (stop < last) {
    Cursor e;
    seek(e, cu, idx, request_of(cu, B, stop), N, pool, state != nullptr);
    stop = owned_from<W>(stop, e);
  }
  float w[W][VEC], b[VEC];
  load_weights<VEC, W>(weight, bias, c, w, b);
  int64_t ld;
  T* const out = out_place<T>(outs, c, ld);

  float win[W - 1][VEC];  // the W - 1 rows before token t, oldest first
  while (t < stop) {
    if (t >= q.end) {
      int64_t r = q.req + 1;
      while (r < B - 1 && cu[r + 1] <= t) ++r;
      if (r >= B) return;
      seek(q, cu, idx, r, N, pool, state != nullptr);
    }
    const int64_t run_end = q.end < stop ? q.end : stop;
    if (run_end <= t || t < q.begin) return;  // cu_seqlens breaks its precondition
    if (!q.live) {
      t = run_end;
      continue;
    }
    const int64_t pos = t - q.begin;
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
      load_row<T, VEC, W>(x, x_stride, state, ch, c, q, pos - (W - 1) + i, win[i]);
    if (pos == 0 && state) {
      const int64_t L = q.end - q.begin;
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int64_t p = L - (W - 1) + i;
        float r[VEC];
        if (p >= 0) {
          load_vec<VEC>(x + (q.begin + p) * x_stride + c, r);
        } else {  // L < W - 1: a history row moves up
#pragma unroll
          for (int k = 0; k < W - 1; ++k)
            if (k == (W - 1) + p)
#pragma unroll
              for (int e = 0; e < VEC; ++e) r[e] = win[k][e];
        }
        store_vec<VEC>(state + (q.slot * (W - 1) + i) * (int64_t)ch + c, r);
      }
    }
    const T* xp = x + t * x_stride + c;
    T* op = out + t * ld;
    auto token = [&](const Raw<T, VEC>& cur, T* to) {
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float now = cur[e];
        float a = b[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) a = __builtin_fmaf(w[j][e], win[j][e], a);
        a = __builtin_fmaf(w[W - 1][e], now, a);
        y[e] = SILU ? a * sigmoidf(a) : a;
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
        win[W - 2][e] = now;
      }
      store_vec<VEC>(to, y);
    };
    // Rows in flight, as they are stored: 33860 tokens of 8192 channels take 317 us with one row
    // converted at its load, 231 with four kept in bf16, 221 with eight.
    constexpr int U = 8;
    Raw<T, VEC> cur[U];
    for (; t + U <= run_end; t += U, xp += U * x_stride, op += U * ld) {
#pragma unroll
      for (int u = 0; u < U; ++u) cur[u].load(xp + u * x_stride);
#pragma unroll
      for (int u = 0; u < U; ++u) token(cur[u], op + u * ld);
    }
    for (; t < run_end; ++t, xp += x_stride, op += ld) {
      cur[0].load(xp);
      token(cur[0], op);
    }
  }
}

// One token per request: the window is the pool's rows, which move up by one.
template <typename T, int VEC, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_decode_kernel(
    const T* __restrict__ x, int64_t x_stride, const float* __restrict__ weight,
    const float* __restrict__ bias, T* __restrict__ state, const int64_t* __restrict__ idx,
    Outs outs, int64_t B, int64_t pool, int per) {
  const int ch = outs.ch;
  const int c = (int)(blockIdx.y * kThreads + threadIdx.x) * VEC;
  if (c >= ch) return;
  float w[W][VEC], b[VEC];
  load_weights<VEC, W>(weight, bias, c, w, b);
  int64_t ld;
  T* const out = out_place<T>(outs, c, ld);
  const int64_t r0 = (int64_t)blockIdx.x * per;
  const int64_t r1 = r0 + per < B ? r0 + per : B;
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t slot = idx[r];
    if (slot < 0 || slot >= pool) continue;  // a padding row
    T* const sp = state + slot * (W - 1) * (int64_t)ch + c;
    float row[W][VEC], y[VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) load_vec<VEC>(sp + i * (int64_t)ch, row[i]);
    load_vec<VEC>(x + r * x_stride + c, row[W - 1]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float a = b[e];
#pragma unroll
      for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][e], row[j][e], a);
      y[e] = SILU ? a * sigmoidf(a) : a;
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_vec<VEC>(sp + i * (int64_t)ch, row[i + 1]);
    store_vec<VEC>(out + r * ld, y);
  }
}

// ---- gradients

// Workgroup of the backward: kCols threads along the channels, kRuns runs of tokens. A thread
// holds weights, their gradients, the window and the g of W tokens for each of its channels:
// four channels leave room for four waves on a SIMD, eight (16 bytes of bf16) for one.
constexpr int kVecBwd = 4;
constexpr int kCols = 64, kRuns = kThreads / kCols;

template <typename T, typename TG, int VEC, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(
    const T* __restrict__ x, int64_t x_stride, const float* __restrict__ weight,
    const float* __restrict__ bias, const T* __restrict__ state, const int64_t* __restrict__ idx,
    const int64_t* __restrict__ cu, Outs dout, const float* __restrict__ dstate,
    T* __restrict__ dx, int64_t dx_stride, float* __restrict__ partial, int64_t N, int64_t B,
    int64_t pool, int run) {
  const int ch = dout.ch;
  const int col = threadIdx.x % kCols, lane_run = threadIdx.x / kCols;
  const int c = (int)(blockIdx.y * kCols + col) * VEC;
  const bool active = c < ch;
  float dw[W][VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  if (active) {
    const int64_t last = cu[B] < N ? cu[B] : N;
    int64_t t = ((int64_t)blockIdx.x * kRuns + lane_run) * run;
    int64_t stop = t + run < last ? t + run : last;
    if (t < cu[0]) t = cu[0];
    if (t < stop) {
      float w[W][VEC], b[VEC];
      load_weights<VEC, W>(weight, bias, c, w, b);
      int64_t ld;
      const TG* const dy = out_place<const TG>(dout, c, ld);
      Cursor q;
      int64_t req = request_of(cu, B, t);
      while (t < stop) {
        seek(q, cu, idx, req, N, pool, state != nullptr);
        if (t < q.begin) break;  // cu_seqlens breaks its precondition
        const int64_t run_end = q.end < stop ? q.end : stop;
        if (q.live && run_end > t) {
          // Token by token: g[p] and its window are formed for the run's tokens and the W - 1
          // after it in the request; dx of a token follows W - 1 tokens behind.
          const int64_t far = run_end + (W - 1) < q.end ? run_end + (W - 1) : q.end;
          float win[W - 1][VEC], g[W][VEC];
#pragma unroll
          for (int i = 0; i < W - 1; ++i)
            load_row<T, VEC, W>(x, x_stride, state, ch, c, q, t - q.begin - (W - 1) + i, win[i]);
#pragma unroll
          for (int i = 0; i < W; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[i][e] = 0.f;
          auto token = [&](int64_t k, const Raw<T, VEC>& xr, const Raw<TG, VEC>& dr) {
            const bool in = k < far, own = k < run_end;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float cur = xr[e];
              float d = in ? dr[e] : 0.f;
              if constexpr (SILU) {
                float a = b[e];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) a = __builtin_fmaf(w[j][e], win[j][e], a);
                a = __builtin_fmaf(w[W - 1][e], cur, a);
                const float sg = sigmoidf(a);
                d = in ? d * (sg * __builtin_fmaf(a, 1.f - sg, 1.f)) : 0.f;
              }
#pragma unroll
              for (int i = 0; i < W - 1; ++i) g[i][e] = g[i + 1][e];
              g[W - 1][e] = d;
              const float go = own ? d : 0.f;
              db[e] += go;
              if (own) {  // rows past the run's end may be another request's
#pragma unroll
                for (int j = 0; j < W - 1; ++j) dw[j][e] = __builtin_fmaf(go, win[j][e], dw[j][e]);
                dw[W - 1][e] = __builtin_fmaf(go, cur, dw[W - 1][e]);
              }
#pragma unroll
              for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
              win[W - 2][e] = cur;
            }
            const int64_t o = k - (W - 1);  // g[s] belongs to token o + s
            if (o >= t) {
              float r[VEC];
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                float a = 0.f;
#pragma unroll
                for (int s = 0; s < W; ++s) a = __builtin_fmaf(w[W - 1 - s][e], g[s][e], a);
                r[e] = a;
              }
              const int64_t srow = o - (q.end - (W - 1));  // its place in the final state
              if (dstate && srow >= 0) {
                float ds[VEC];
                load_vec<VEC>(dstate + (q.req * (W - 1) + srow) * (int64_t)ch + c, ds);
#pragma unroll
                for (int e = 0; e < VEC; ++e) r[e] += ds[e];
              }
              store_vec<VEC>(dx + o * dx_stride + c, r);
            }
          };
          constexpr int U = 4;  // rows in flight; the last rows of a request are read again
          const int64_t kend = run_end + (W - 1);
          for (int64_t k = t; k < kend; k += U) {
            Raw<T, VEC> xr[U];
            Raw<TG, VEC> dr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int64_t kk = k + u < far ? k + u : far - 1;
              xr[u].load(x + kk * x_stride + c);
              dr[u].load(dy + kk * ld);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (k + u < kend) token(k + u, xr[u], dr[u]);
          }
        }
        if (run_end > t) t = run_end;
        ++req;
        if (req >= B) break;
      }
    }
  }
  // the runs of the workgroup, added in a fixed order; one partial row per workgroup
  __shared__ float s_red[kRuns][kCols * VEC];
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      s_red[lane_run][col * VEC + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int k = threadIdx.x; k < kCols * VEC; k += kThreads) {
      float a = 0.f;
#pragma unroll
      for (int r = 0; r < kRuns; ++r) a += s_red[r][k];
      const int cc = (int)blockIdx.y * kCols * VEC + k;
      if (cc < ch) partial[((int64_t)blockIdx.x * (W + 1) + j) * ch + cc] = a;
    }
  }
}

// dweight and dbias: the workgroups' partial rows [blocks][W + 1][ch], added in order.
__global__ __launch_bounds__(kThreads) void conv_bwd_sum_kernel(
    const float* __restrict__ partial, int64_t blocks, int W, int ch, float* __restrict__ dweight,
    float* __restrict__ dbias) {
  constexpr int C = 32, R = kThreads / C;
  __shared__ float s_red[R][C];
  const int col = threadIdx.x % C, r = threadIdx.x / C;
  const int c = (int)blockIdx.x * C + col, j = blockIdx.y;
  float a = 0.f;
  if (c < ch)
    for (int64_t k = r; k < blocks; k += R) a += partial[(k * (W + 1) + j) * ch + c];
  s_red[r][col] = a;
  __syncthreads();
  if (r == 0 && c < ch) {
#pragma unroll
    for (int i = 1; i < R; ++i) a += s_red[i][col];
    if (j < W)
      dweight[(int64_t)c * W + j] = a;
    else if (dbias)
      dbias[c] = a;
  }
}

// dstate0: du of the history rows, e = i - (W - 1) < 0, from the first W - 1 tokens' g.
template <typename T, typename TG, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_bwd_state_kernel(
    const T* __restrict__ x, int64_t x_stride, const float* __restrict__ weight,
    const float* __restrict__ bias, const T* __restrict__ state, const int64_t* __restrict__ idx,
    const int64_t* __restrict__ cu, Outs dout, const float* __restrict__ dstate,
    float* __restrict__ dstate0, int64_t N, int64_t pool) {
  const int ch = dout.ch;
  const int c = (int)(blockIdx.y * kThreads + threadIdx.x);
  if (c >= ch) return;
  const int64_t req = blockIdx.x;
  Cursor q;
  seek(q, cu, idx, req, N, pool, state != nullptr);
  float du[W - 1];
#pragma unroll
  for (int i = 0; i < W - 1; ++i) du[i] = 0.f;
  if (q.live) {
    const int64_t L = q.end > q.begin ? q.end - q.begin : 0;
    float w[W][1], b[1];
    load_weights<1, W>(weight, bias, c, w, b);
    int64_t ld;
    const TG* const dy = out_place<const TG>(dout, c, ld);
    float u[2 * (W - 1)][1];
#pragma unroll
    for (int i = 0; i < 2 * (W - 1); ++i) {
      u[i][0] = 0.f;
      if (i - (W - 1) < L)
        load_row<T, 1, W>(x, x_stride, state, ch, c, q, i - (W - 1), u[i]);
    }
#pragma unroll
    for (int p = 0; p < W - 1; ++p) {
      if (p >= L) break;
      float g = (float)dy[(q.begin + p) * ld];
      if constexpr (SILU) {
        float a = b[0];
#pragma unroll
        for (int j = 0; j < W; ++j) a = __builtin_fmaf(w[j][0], u[p + j][0], a);
        const float sg = sigmoidf(a);
        g *= sg * __builtin_fmaf(a, 1.f - sg, 1.f);
      }
#pragma unroll
      for (int i = p; i < W - 1; ++i) du[i] = __builtin_fmaf(w[i - p][0], g, du[i]);
    }
    if (dstate) {  // L < W - 1: the newest history rows stay in the final state
#pragma unroll
      for (int i = 0; i < W - 1; ++i)
        if (i >= L) du[i] += dstate[(req * (W - 1) + (i - L)) * (int64_t)ch + c];
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) dstate0[(req * (W - 1) + i) * (int64_t)ch + c] = du[i];
}

// Tokens of a tile: long enough that the window's rows, which mostly hit in L2, are a small share
// of what a tile reads, short enough that a small call still spreads over the device.
int fwd_tile(const ConvShape& s, int vec) {
  const int64_t cols = cdiv(cdiv(s.ch, vec), kThreads);
  int tile = 32;
  while (tile > 4 && cdiv(s.N, tile) * cols < 1024) tile /= 2;
  return tile;
}

int bwd_run(const ConvShape& s, int vec) {
  const int64_t cols = cdiv(cdiv(s.ch, vec), kCols);
  int run = 128;
  while (run > 8 && cdiv(s.N, (int64_t)run * kRuns) * cols < 512) run /= 2;
  return run;
}

// Requests of a thread of the single-token kernel: with enough of them to fill the device several
// are taken in turn, so that the weights, more bytes than a token's, are loaded once for them
// (512 requests of 8192 channels: 16.2, 13.8 and 12.6 us with 1, 2 and 4).
int decode_requests(const ConvShape& s, int64_t cols) {
  const int64_t n = s.B * cols / 512;
  return n < 1 ? 1 : n > 4 ? 4 : (int)n;
}

int vec_of(const ConvShape& s) { return s.vec ? (s.bf16 ? 8 : 4) : 1; }
int vec_bwd(const ConvShape& s) { return s.vec ? kVecBwd : 1; }

template <typename T, int VEC, int W, bool SILU>
hipError_t conv_fwd_t(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      void* state, const int64_t* idx, const int64_t* cu, const Outs& o,
                      bool decode, hipStream_t st) {
  const unsigned cols = (unsigned)cdiv(cdiv(s.ch, VEC), kThreads);
  if (decode) {
    const int per = decode_requests(s, cols);
    hipLaunchKernelGGL((conv_decode_kernel<T, VEC, W, SILU>),
                       dim3((unsigned)cdiv(s.B, per), cols), dim3(kThreads), 0, st, (const T*)x,
                       s.x_stride, weight, bias, (T*)state, idx, o, s.B, s.pool, per);
  } else {
    const int tile = fwd_tile(s, VEC);
    hipLaunchKernelGGL((conv_fwd_kernel<T, VEC, W, SILU>), dim3((unsigned)cdiv(s.N, tile), cols),
                       dim3(kThreads), 0, st, (const T*)x, s.x_stride, weight, bias, (T*)state,
                       idx, cu, o, s.N, s.B, s.pool, tile);
  }
  return hipGetLastError();
}

template <typename T, typename TG, int VEC, int W, bool SILU>
hipError_t conv_bwd_t(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      const void* state, const int64_t* idx, const int64_t* cu, const Outs& dout,
                      const float* dstate, void* dx, float* dweight, float* dbias,
                      float* dstate0, float* ws, hipStream_t st) {
  const int run = bwd_run(s, VEC);
  const int64_t blocks = cdiv(s.N, (int64_t)run * kRuns);
  if (blocks > 0) {
    hipLaunchKernelGGL((conv_bwd_kernel<T, TG, VEC, W, SILU>),
                       dim3((unsigned)blocks, (unsigned)cdiv(cdiv(s.ch, VEC), kCols)),
                       dim3(kThreads), 0, st, (const T*)x, s.x_stride, weight, bias,
                       (const T*)state, idx, cu, dout, dstate, (T*)dx, s.dx_stride, ws, s.N, s.B,
                       s.pool, run);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((unsigned)cdiv(s.ch, 32), (unsigned)(W + 1)),
                     dim3(kThreads), 0, st, ws, blocks, W, s.ch, dweight, dbias);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (dstate0) {
    hipLaunchKernelGGL((conv_bwd_state_kernel<T, TG, W, SILU>),
                       dim3((unsigned)s.B, (unsigned)cdiv(s.ch, kThreads)), dim3(kThreads), 0, st,
                       (const T*)x, s.x_stride, weight, bias, (const T*)state, idx, cu, dout,
                       dstate, dstate0, s.N, s.pool);
    return hipGetLastError();
  }
  return hipSuccess;
}

template <typename T, int VEC, int W>
hipError_t conv_fwd_w(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      void* state, const int64_t* idx, const int64_t* cu, const Outs& o,
                      bool decode, hipStream_t st) {
  return s.silu ? conv_fwd_t<T, VEC, W, true>(s, x, weight, bias, state, idx, cu, o, decode, st)
                : conv_fwd_t<T, VEC, W, false>(s, x, weight, bias, state, idx, cu, o, decode, st);
}

template <typename T, int VEC>
hipError_t conv_fwd_v(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      void* state, const int64_t* idx, const int64_t* cu, const Outs& o,
                      bool decode, hipStream_t st) {
  switch (s.W) {
    case 2: return conv_fwd_w<T, VEC, 2>(s, x, weight, bias, state, idx, cu, o, decode, st);
    case 3: return conv_fwd_w<T, VEC, 3>(s, x, weight, bias, state, idx, cu, o, decode, st);
    case 4: return conv_fwd_w<T, VEC, 4>(s, x, weight, bias, state, idx, cu, o, decode, st);
  }
  return hipErrorInvalidValue;
}

hipError_t conv_fwd_any(const ConvShape& s, const void* x, const float* weight,
                        const float* bias, void* state, const int64_t* idx, const int64_t* cu,
                        void* const out[3], bool decode, hipStream_t st) {
  const Outs o{{out[0], out[1], out[2]}, s.c1, s.c2, s.ch};
  if (s.bf16)
    return s.vec ? conv_fwd_v<__bf16, 8>(s, x, weight, bias, state, idx, cu, o, decode, st)
                 : conv_fwd_v<__bf16, 1>(s, x, weight, bias, state, idx, cu, o, decode, st);
  return s.vec ? conv_fwd_v<float, 4>(s, x, weight, bias, state, idx, cu, o, decode, st)
               : conv_fwd_v<float, 1>(s, x, weight, bias, state, idx, cu, o, decode, st);
}

template <typename T, typename TG, int VEC, int W>
hipError_t conv_bwd_w(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      const void* state, const int64_t* idx, const int64_t* cu, const Outs& dout,
                      const float* dstate, void* dx, float* dweight, float* dbias,
                      float* dstate0, float* ws, hipStream_t st) {
  return s.silu ? conv_bwd_t<T, TG, VEC, W, true>(s, x, weight, bias, state, idx, cu, dout,
                                                  dstate, dx, dweight, dbias, dstate0, ws, st)
                : conv_bwd_t<T, TG, VEC, W, false>(s, x, weight, bias, state, idx, cu, dout,
                                                   dstate, dx, dweight, dbias, dstate0, ws, st);
}

template <typename T, typename TG, int VEC>
hipError_t conv_bwd_v(const ConvShape& s, const void* x, const float* weight, const float* bias,
                      const void* state, const int64_t* idx, const int64_t* cu, const Outs& dout,
                      const float* dstate, void* dx, float* dweight, float* dbias,
                      float* dstate0, float* ws, hipStream_t st) {
  switch (s.W) {
    case 2: return conv_bwd_w<T, TG, VEC, 2>(s, x, weight, bias, state, idx, cu, dout, dstate, dx,
                                             dweight, dbias, dstate0, ws, st);
    case 3: return conv_bwd_w<T, TG, VEC, 3>(s, x, weight, bias, state, idx, cu, dout, dstate, dx,
                                             dweight, dbias, dstate0, ws, st);
    case 4: return conv_bwd_w<T, TG, VEC, 4>(s, x, weight, bias, state, idx, cu, dout, dstate, dx,
                                             dweight, dbias, dstate0, ws, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool conv_grids_fit(const ConvShape& s, bool backward) {
  const int vec = backward ? vec_bwd(s) : vec_of(s);
  const int64_t cols = cdiv(s.ch, (int64_t)vec * (backward ? kCols : kThreads));
  const int64_t x = backward ? cdiv(s.N, (int64_t)bwd_run(s, vec) * kRuns)
                             : cdiv(s.N, fwd_tile(s, vec));
  return cols <= 65535 && cdiv(s.ch, kThreads) <= 65535 && grid_ok(x, kThreads) &&
         grid_ok(s.B, kThreads);
}

hipError_t launch_conv_fwd(const ConvShape& s, const void* x, const float* weight,
                           const float* bias, void* state, const int64_t* idx, const int64_t* cu,
                           void* const out[3], hipStream_t st) {
  return conv_fwd_any(s, x, weight, bias, state, idx, cu, out, false, st);
}

hipError_t launch_conv_decode(const ConvShape& s, const void* x, const float* weight,
                              const float* bias, void* state, const int64_t* idx,
                              void* const out[3], hipStream_t st) {
  return conv_fwd_any(s, x, weight, bias, state, idx, nullptr, out, true, st);
}

size_t conv_bwd_workspace(const ConvShape& s) {
  // whichever path serves the call: vectors have fewer column blocks, hence shorter runs and, up to
  // four times, more partial rows
  ConvShape t = s;
  size_t rows = 0;
  for (const bool vec : {false, true}) {
    t.vec = vec;
    const size_t r = (size_t)cdiv(s.N, (int64_t)bwd_run(t, vec_bwd(t)) * kRuns);
    rows = r > rows ? r : rows;
  }
  return align256(rows * (size_t)(s.W + 1) * (size_t)s.ch * sizeof(float));
}

hipError_t launch_conv_bwd(const ConvShape& s, const void* x, const float* weight,
                           const float* bias, const void* state, const int64_t* idx,
                           const int64_t* cu, const void* const dout[3], const float* dstate,
                           void* dx, float* dweight, float* dbias, float* dstate0, float* ws,
                           hipStream_t st) {
  const Outs o{{const_cast<void*>(dout[0]), const_cast<void*>(dout[1]),
                const_cast<void*>(dout[2])}, s.c1, s.c2, s.ch};
#define GDN_CONV_BWD(T, TG, VEC) \
  return conv_bwd_v<T, TG, VEC>(s, x, weight, bias, state, idx, cu, o, dstate, dx, dweight, \
                                dbias, dstate0, ws, st)
  if (s.bf16) {
    if (s.dout_bf16) {
      if (s.vec) GDN_CONV_BWD(__bf16, __bf16, kVecBwd);
      GDN_CONV_BWD(__bf16, __bf16, 1);
    }
    if (s.vec) GDN_CONV_BWD(__bf16, float, kVecBwd);
    GDN_CONV_BWD(__bf16, float, 1);
  }
  if (s.dout_bf16) {
    if (s.vec) GDN_CONV_BWD(float, __bf16, 4);
    GDN_CONV_BWD(float, __bf16, 1);
  }
  if (s.vec) GDN_CONV_BWD(float, float, 4);
  GDN_CONV_BWD(float, float, 1);
#undef GDN_CONV_BWD
}

}  // namespace layer
}  // namespace gdn
