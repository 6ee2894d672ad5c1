// Selective state space scan over packed requests, chunk by chunk on the matrix cores.
//
// With g_t = log a_t = -exp(A_log) d_t, d_t = softplus(dt + dt_bias), G the running sum of g in
// a chunk and S the state before it (dv x dk):
//   y_t  = e^{G_t} S C_t + sum_{j <= t} e^{G_t - G_j} d_j (C_t . B_j) x_j + D x_t
//   S   <- e^{G_n} S + sum_t (e^{G_n - G_t} d_t x_t) B_t^T
// Unlike the delta rule nothing has to be inverted: a chunk is four products (scores C B^T, scores
// times x, S C, x B^T), all in 16x16x32 matrix instructions with fp32 sums.
//
// A workgroup of four waves walks the chunks of one segment of a request for 128 of the value
// columns that share a group's B and C (the group's heads side by side, 32 columns of one head
// per wave). A wave keeps its 32 columns of S^T (dk x 32, fp32) in registers from the first
// chunk to the last. In the D layout of the products a lane holds four consecutive state entries
// of one column, which is also what the next products want as an operand, so the state and the
// scores never move between lanes.
//
// Requests longer than a segment are cut: a first pass forms each segment's state from zero, a
// second joins them in order into every segment's start state, and the output pass runs all
// segments side by side. Only the scalar decay per head lies between two segments, so the join
// is one multiply-add per state entry and segment.
//
// Precision: bf16 inputs enter the products as they are. The decayed x of the state's update are
// pairs of bf16 (hi + lo, at most 2^-17 off), since states are fp32 results; the decayed scores
// and the state that S C reads are one bf16 each (2^-8 of a term: the output is rounded by as
// much). For fp32 inputs every operand is three bf16 (24 bits) and a product takes the six pairs
// of parts that reach 2^-24: 2.7 times the rate of the fp32 matrix instructions.
// Gates and their sums are fp32 (the sums of fp32 inputs fp64), and exponents are only taken of
// differences that are not positive, so strong decays underflow to zero and nothing overflows.
#include "gdn_layer.h"
#include "gdn_mfma.h"

namespace gdn {
namespace layer {
namespace {

using mfma::bf16x8_from_u32x4;
using mfma::kperm;
using mfma::mma_bf16;
using mfma::u32x2;
using mfma::u32x4;
typedef mfma::bf16x8 bfrag;
typedef mfma::f32x4 acc4;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kColsWave = 32, kColsBlock = kColsWave * kWaves;  // value columns
constexpr int kPad = 8;  // bf16 entries between LDS rows: the rows of a fragment in other banks

struct ScanArgs {
  const void *C, *B, *x;
  const float *dt, *A_log, *dt_bias, *D;
  float* pool;
  const int64_t *idx, *cu;
  void* out;
  float* seg_state;   // [segments of cut requests][HV][dv][dk]
  float* seg_decay;   // [segments of cut requests][HV]: sum of g over the segment
  int64_t N, nreq, npool;
  int H, HV, dv, rep, blocks_per_group;
  int lseg;           // tokens of a segment (a multiple of 64), 0: nothing is cut
  int max_cut;        // places in seg_state
};

// Segments of a request of L tokens (an empty request counts one, which has nothing to do).
__device__ __forceinline__ int segments_of(int64_t L, int lseg) {
  return lseg == 0 || L <= lseg ? 1 : (int)((L + lseg - 1) / lseg);
}

__device__ __forceinline__ int64_t begin_of(const ScanArgs& a, int64_t b) {
  return a.cu[b] < 0 ? 0 : a.cu[b];
}
__device__ __forceinline__ int64_t end_of(const ScanArgs& a, int64_t b) {
  return a.cu[b + 1] < a.N ? a.cu[b + 1] : a.N;
}

struct Segment {
  int64_t req;
  int64_t t0, t1;  // tokens
  int index, count;  // of its request
  int ws;  // place among the segments of cut requests (cut requests only)
};

__device__ __forceinline__ int wave_inclusive(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(v, off, 64);
    if (lane >= off) v += y;
  }
  return v;
}

// Segment number `seg` of the call, by a scan over the requests, 64 at a time in every wave.
__device__ __forceinline__ bool find_segment(const ScanArgs& a, int seg, Segment& s) {
  const int lane = threadIdx.x & 63;
  if (a.lseg == 0) {
    s.req = seg;
    s.index = 0;
    s.count = 1;
    s.ws = 0;
  } else {
    int before = 0, before_cut = 0;
    bool found = false;
    for (int64_t base = 0; base < a.nreq; base += 64) {
      const int64_t b = base + lane;
      const int n = b < a.nreq ? segments_of(end_of(a, b) - begin_of(a, b), a.lseg) : 0;
      const int inc = wave_inclusive(n), cut = wave_inclusive(n > 1 ? n : 0);
      const uint64_t over = __ballot(before + inc > seg);
      if (over) {
        const int k = __builtin_ctzll(over);
        s.count = __builtin_amdgcn_readlane(n, k);
        s.index = seg - before - (__builtin_amdgcn_readlane(inc, k) - s.count);
        s.ws = before_cut + __builtin_amdgcn_readlane(cut, k) - s.count + s.index;
        s.req = base + k;
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(inc, 63);
      before_cut += __builtin_amdgcn_readlane(cut, 63);
    }
    if (!found) return false;
  }
  const int64_t begin = begin_of(a, s.req), end = end_of(a, s.req);
  s.t0 = begin + (int64_t)s.index * a.lseg;
  s.t1 = s.index + 1 < s.count ? s.t0 + a.lseg : end;
  const int64_t slot = a.idx[s.req];
  if (s.count > 1 && s.ws >= a.max_cut) return false;  // cu_seqlens breaks its precondition
  return s.t0 < s.t1 && slot >= 0 && slot < a.npool;
}

__device__ __forceinline__ float softplusf(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// v as a sum of P bf16: 2^-8, 2^-17 or 2^-25 of v off.
template <int P>
__device__ __forceinline__ void split(float v, __bf16 (&part)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    part[p] = (__bf16)v;
    v -= (float)part[p];
  }
}

// Running sums over the wave's lanes, inclusive from the front, exclusive from the back.
template <typename R>
__device__ __forceinline__ R prefix(R v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const R y = __shfl_up(v, off, 64);
    if (lane >= off) v += y;
  }
  return v;
}
__device__ __forceinline__ float suffix_exclusive(float g) {
  const int lane = threadIdx.x & 63;
  float v = __shfl_down(g, 1, 64);
  if (lane == 63) v = 0.f;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const float y = __shfl_down(v, off, 64);
    if (lane + off < 64) v += y;
  }
  return v;
}

// What a wave knows of a chunk's gates, one entry per token (its own head's).
template <int CH, typename R>
struct Gates {
  R G[CH];             // running sum of g in the chunk
  float step[CH];      // d
  float eG[CH];        // e^G
  float row[CH];       // e^{G_t - G at the start of t's tile}
  float w[CH];         // d e^{G_n - G}: weight in the state's update
  float col[CH / 16][CH];  // [tile]: d_j e^{G at the tile's start - G_j}, j before the tile
};

// Eight entries of a row at k = kperm(g, 0..7), two 8-byte reads.
__device__ __forceinline__ bfrag frag_kperm(const __bf16* row, int g) {
  const u32x2 lo = *reinterpret_cast<const u32x2*>(row + 4 * g);
  const u32x2 hi = *reinterpret_cast<const u32x2*>(row + 16 + 4 * g);
  return bf16x8_from_u32x4(u32x4{lo[0], lo[1], hi[0], hi[1]});
}
// Column col0 + m of a row-major tile, rows 32 s + kperm(g, 0..7).
__device__ __forceinline__ bfrag frag_col(const __bf16* tile, int ld, int col0, int s, int g, int m) {
  return bf16x8_from_u32x4(
      mfma::col_frag_tr(reinterpret_cast<const uint16_t*>(tile), ld, col0, s, g, m));
}

// Staging of a tile of CH rows x COLS entries: 16-byte pieces in registers between the load and
// the LDS store, so that the next chunk's rows travel while this one is worked on.
template <typename T, int CH, int COLS>
struct Stage {
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int PER_ROW = COLS / V, PIECES = CH * PER_ROW / kThreads;
  static_assert(CH * PER_ROW % kThreads == 0, "whole pieces per thread");
  u32x4 r[PIECES];
  // rows t0 .. t0 + CH - 1 of a matrix with row stride ld; rows from t1 on, and columns from
  // `cols` on, read as zero
  __device__ __forceinline__ void load(const T* base, int64_t ld, int64_t t0, int64_t t1, int cols) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = i * kThreads + threadIdx.x, row = p / PER_ROW, c = p % PER_ROW * V;
      r[i] = u32x4{0, 0, 0, 0};
      if (t0 + row < t1 && c < cols)
        r[i] = *reinterpret_cast<const u32x4*>(base + (t0 + row) * ld + c);
    }
  }
  // as NP tiles of bf16 parts, `plane` entries apart
  template <int NP>
  __device__ __forceinline__ void store(__bf16* to, int plane, int ld) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = i * kThreads + threadIdx.x, row = p / PER_ROW, c = p % PER_ROW * V;
      if constexpr (NP == 1) {
        *reinterpret_cast<u32x4*>(to + row * ld + c) = r[i];
      } else {
        const f32x4 v = __builtin_bit_cast(f32x4, r[i]);
        bf16x4 part[NP];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          __bf16 one[NP];
          split<NP>(v[e], one);
#pragma unroll
          for (int p = 0; p < NP; ++p) part[p][e] = one[p];
        }
#pragma unroll
        for (int p = 0; p < NP; ++p)
          *reinterpret_cast<bf16x4*>(to + p * plane + row * ld + c) = part[p];
      }
    }
  }
};

// The tiles of the lower triangle of CH / 16 x CH / 16 tiles, row by row.
__device__ __forceinline__ void triangle(int i, int& tt, int& jt) {
  tt = i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3;
  jt = i - tt * (tt + 1) / 2;
}

// OUT: the output pass. Otherwise the pass that forms each segment's state from zero.
template <typename T, int DK, int CH, bool OUT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void ssm_scan_kernel(ScanArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int NP = F32 ? 3 : 1;               // bf16 parts of an input, scores and S in S C
  constexpr int NU = F32 ? 3 : 2;               // ... of the update's decayed x
  constexpr int NT = CH / 16, NK = CH / 32;      // token tiles, k steps over tokens
  constexpr int NS = DK / 16, NKS = DK / 32;     // state tiles, k steps over state entries
  constexpr int LDB = DK + kPad, LDX = kColsBlock + kPad, LDR = CH + 4;
  constexpr int NTRI = NT * (NT + 1) / 2, TRI = (NTRI + kWaves - 1) / kWaves;
  using R = typename std::conditional<F32, double, float>::type;
  using G = Gates<CH, R>;

  constexpr int kTileB = CH * LDB, kTileX = CH * LDX;
  // the scores take C's place once S C has been formed
  constexpr int kC = !OUT ? 0 : kTileB * NP * 2 > CH * LDR * 4 ? kTileB * NP * 2 : CH * LDR * 4;
  __shared__ __align__(16) char s_c[kC + 16];
  __shared__ __align__(16) __bf16 s_b[NP * kTileB];
  __shared__ __align__(16) __bf16 s_x[NP * kTileX];
  __shared__ G s_g[kWaves];
  __bf16* const tc = reinterpret_cast<__bf16*>(s_c);
  float* const raw = reinterpret_cast<float*>(s_c);

  const int blk = blockIdx.x;
  const int per_seg = a.H * a.blocks_per_group;
  Segment sg;
  if (!find_segment(a, blk / per_seg, sg)) return;
  const bool last = sg.index + 1 == sg.count;
  if (!OUT && last) return;  // nothing starts from it
  const int in_seg = blk % per_seg, h = in_seg / a.blocks_per_group;
  const int col0 = in_seg % a.blocks_per_group * kColsBlock;  // of the group's columns
  const int vc = a.rep * a.dv;
  const int ncols = vc - col0 < kColsBlock ? vc - col0 : kColsBlock;

  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, g = lane >> 4;
  const bool live = kColsWave * wv < ncols;
  const int wcol = live ? col0 + kColsWave * wv : col0;
  const int hv = h * a.rep + wcol / a.dv, p0 = wcol % a.dv;
  const int64_t slot = a.idx[sg.req];

  const T* const gB = reinterpret_cast<const T*>(a.B) + (int64_t)h * DK;
  const T* const gC = reinterpret_cast<const T*>(a.C) + (int64_t)h * DK;
  const T* const gx = reinterpret_cast<const T*>(a.x) + (int64_t)h * vc + col0;
  const int64_t ldb = (int64_t)a.H * DK, ldx = (int64_t)a.HV * a.dv;

  // S^T: st[s tile][column tile], entries 16 s + 4 g .. + 3 of column p0 + 16 pt + r
  acc4 st[NS][2];
  const float* from = nullptr;
  const int64_t plane = (int64_t)a.dv * DK;
  if (OUT) {
    from = sg.count > 1 ? a.seg_state + ((int64_t)sg.ws * a.HV + hv) * plane
                        : a.pool + (slot * a.HV + hv) * plane;
    from += (int64_t)(p0 + r) * DK + 4 * g;
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
      st[s][pt] = OUT && live ? *reinterpret_cast<const acc4*>(from + 16 * pt * DK + 16 * s)
                              : acc4{0.f, 0.f, 0.f, 0.f};

  const float decay = -expf(a.A_log[hv]), dtb = a.dt_bias[hv];
  const float dskip = a.D ? a.D[hv] : 0.f;
  float gsum = 0.f;  // of g over the segment

  Stage<T, CH, DK> qb, qc;
  Stage<T, CH, kColsBlock> qx;
  float qdt = 0.f;
  auto fetch = [&](int64_t t) {
    qb.load(gB, ldb, t, sg.t1, DK);
    if constexpr (OUT) qc.load(gC, ldb, t, sg.t1, DK);
    qx.load(gx, ldx, t, sg.t1, ncols);
    qdt = lane < CH && t + lane < sg.t1 ? a.dt[(t + lane) * a.HV + hv] : 0.f;
  };
  fetch(sg.t0);

  for (int64_t t0 = sg.t0; t0 < sg.t1; t0 += CH) {
    if (t0 > sg.t0) __syncthreads();  // the chunk before has been read
    qb.template store<NP>(s_b, kTileB, LDB);
    if constexpr (OUT) qc.template store<NP>(tc, kTileB, LDB);
    qx.template store<NP>(s_x, kTileX, LDX);
    G& gt = s_g[wv];
    float eGn;
    {  // gates, a lane per token; rows past the end have no step and no decay
      const bool in = lane < CH && t0 + lane < sg.t1;
      const float step = in ? softplusf(qdt + dtb) : 0.f;
      const float gl = in ? decay * step : 0.f;
      const R Gp = prefix<R>((R)gl);
      const float rest = suffix_exclusive(gl);
      const float tot = (float)__shfl(Gp, 63, 64);
      eGn = expf(tot);
      gsum += tot;
      if constexpr (OUT) {
        R at[NT];  // G before each tile
        at[0] = 0;
#pragma unroll
        for (int k = 1; k < NT; ++k) at[k] = __shfl(Gp, 16 * k - 1, 64);
        if (lane < CH) {
          gt.G[lane] = Gp;
          gt.step[lane] = step;
          gt.eG[lane] = expf((float)Gp);
          R mine = at[0];
#pragma unroll
          for (int k = 1; k < NT; ++k) {
            if (lane / 16 == k) mine = at[k];
            gt.col[k][lane] = lane < 16 * k ? step * expf((float)(at[k] - Gp)) : 0.f;
          }
          gt.row[lane] = expf((float)(Gp - mine));
        }
      }
      if (lane < CH) gt.w[lane] = step * expf(rest);
    }
    __syncthreads();
    if (t0 + CH < sg.t1) fetch(t0 + CH);

    bfrag xf[NP][2][NK];  // x, column p0 + 16 pt + r, tokens 32 k + kperm
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int k = 0; k < NK; ++k)
          xf[p][pt][k] = frag_col(s_x + p * kTileX, LDX, kColsWave * wv + 16 * pt, k, g, r);

    if constexpr (OUT) {
      // Y^T = e^G (S C^T): y[t tile][column tile], columns 4 g .. + 3 of token 16 t + r
      acc4 y[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) y[t][pt] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NKS; ++k) {
        bfrag sb[NP][2];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            __bf16 part[NP];
            split<NP>(st[2 * k + e / 4][pt][e % 4], part);
#pragma unroll
            for (int p = 0; p < NP; ++p) sb[p][pt][e] = part[p];
          }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bfrag c = frag_kperm(tc + p * kTileB + (16 * t + r) * LDB + 32 * k, g);
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
              for (int q = 0; q + p < NP; ++q) y[t][pt] = mma_bf16(sb[q][pt], c, y[t][pt]);
          }
      }
      // scores^T, j x t, shared by the workgroup's heads: each wave some of the tiles
      acc4 sc[TRI];
#pragma unroll
      for (int i = 0; i < TRI; ++i) {
        sc[i] = acc4{0.f, 0.f, 0.f, 0.f};
        const int n = wv + i * kWaves;
        if (n >= NTRI) continue;
        int tt, jt;
        triangle(n, tt, jt);
#pragma unroll
        for (int k = 0; k < NKS; ++k)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bfrag c = *reinterpret_cast<const bfrag*>(
                tc + p * kTileB + (16 * tt + r) * LDB + 32 * k + 8 * g);
#pragma unroll
            for (int q = 0; q + p < NP; ++q) {
              const bfrag b = *reinterpret_cast<const bfrag*>(
                  s_b + q * kTileB + (16 * jt + r) * LDB + 32 * k + 8 * g);
              sc[i] = mma_bf16(b, c, sc[i]);
            }
          }
      }
      __syncthreads();  // C has been read
#pragma unroll
      for (int i = 0; i < TRI; ++i) {
        const int n = wv + i * kWaves;
        if (n >= NTRI) continue;
        int tt, jt;
        triangle(n, tt, jt);
        *reinterpret_cast<acc4*>(raw + (16 * tt + r) * LDR + 16 * jt + 4 * g) = sc[i];
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float e = gt.eG[16 * t + r], row = gt.row[16 * t + r];
        const R Gt = gt.G[16 * t + r];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) y[t][pt] *= e;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          if (2 * k > t) continue;
          bfrag pf[NP];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int j = 2 * k + half;  // tile of tokens j
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (j <= t) {
              const acc4 s = *reinterpret_cast<const acc4*>(raw + (16 * t + r) * LDR + 16 * j + 4 * g);
              if (j < t) {
                const acc4 c = *reinterpret_cast<const acc4*>(&gt.col[t][16 * j + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = s[i] * (c[i] * row);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int jj = 16 * j + 4 * g + i;
                  const float ex = expf((float)(Gt - gt.G[jj])) * gt.step[jj];
                  v[i] = 4 * g + i <= r ? s[i] * ex : 0.f;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              __bf16 part[NP];
              split<NP>(v[i], part);
#pragma unroll
              for (int p = 0; p < NP; ++p) pf[p][4 * half + i] = part[p];
            }
          }
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
              for (int q = 0; q + p < NP; ++q)
                y[t][pt] = mma_bf16(xf[p][pt][k], pf[q], y[t][pt]);
        }
        // + D x, and out: four columns of one token per lane
        const int64_t tok = t0 + 16 * t + r;
        if (live && tok < sg.t1) {
#pragma unroll
          for (int pt = 0; pt < 2; ++pt) {
            const int at = (16 * t + r) * LDX + kColsWave * wv + 16 * pt + 4 * g;
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float xv = 0.f;
#pragma unroll
              for (int p = NP - 1; p >= 0; --p) xv += (float)s_x[p * kTileX + at + i];
              o[i] = __builtin_fmaf(dskip, xv, y[t][pt][i]);
            }
            T* const dst = reinterpret_cast<T*>(a.out) + tok * ldx + (int64_t)hv * a.dv + p0 +
                           16 * pt + 4 * g;
            if constexpr (F32) {
              *reinterpret_cast<f32x4*>(dst) = f32x4{o[0], o[1], o[2], o[3]};
            } else {
              *reinterpret_cast<bf16x4*>(dst) =
                  bf16x4{(__bf16)o[0], (__bf16)o[1], (__bf16)o[2], (__bf16)o[3]};
            }
          }
        }
      }
    }

    // S^T <- e^{G_n} S^T + B^T (w x)
    bfrag xw[NU][2][NK];
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float v = 0.f;
#pragma unroll
          for (int p = NP - 1; p >= 0; --p) v += (float)xf[p][pt][k][e];
          __bf16 part[NU];
          split<NU>(v * gt.w[32 * k + kperm(g, e)], part);
#pragma unroll
          for (int p = 0; p < NU; ++p) xw[p][pt][k][e] = part[p];
        }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int pt = 0; pt < 2; ++pt) st[s][pt] *= eGn;
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const bfrag b = frag_col(s_b + p * kTileB, LDB, 16 * s, k, g, r);
#pragma unroll
          for (int pt = 0; pt < 2; ++pt)
#pragma unroll
            for (int q = 0; q + p < NU; ++q)
              // pieces of a cut request but its last: their state is only read by S C above
              if (q == 0 || !OUT || F32 || last) st[s][pt] = mma_bf16(b, xw[q][pt][k], st[s][pt]);
        }
    }
  }

  if (!live || (OUT && !last)) return;
  float* to = OUT ? a.pool + (slot * a.HV + hv) * plane
                  : a.seg_state + ((int64_t)sg.ws * a.HV + hv) * plane;
  to += (int64_t)(p0 + r) * DK + 4 * g;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
      *reinterpret_cast<acc4*>(to + 16 * pt * DK + 16 * s) = st[s][pt];
  if (!OUT && p0 == 0 && lane == 0) a.seg_decay[(int64_t)sg.ws * a.HV + hv] = gsum;
}

// Start states of a cut request's segments, in place of the segments' own states.
__global__ __launch_bounds__(256) void ssm_join_kernel(ScanArgs a, int plane, int parts) {
  const int part = blockIdx.x % parts;
  const int64_t pair = blockIdx.x / parts;
  const int64_t req = pair / a.HV;
  const int hv = (int)(pair - req * a.HV);
  const int64_t slot = a.idx[req];
  const int n = segments_of(end_of(a, req) - begin_of(a, req), a.lseg);
  if (n <= 1 || slot < 0 || slot >= a.npool) return;
  int first = 0;  // place of the request's first segment
  for (int64_t base = 0; base < req; base += 64) {
    const int64_t b = base + (threadIdx.x & 63);
    const int k = b < req ? segments_of(end_of(a, b) - begin_of(a, b), a.lseg) : 0;
    first += __builtin_amdgcn_readlane(wave_inclusive(k > 1 ? k : 0), 63);
  }
  const int e = (part * 256 + threadIdx.x) * 4;
  if (first + n > a.max_cut) return;
  f32x4 s = *reinterpret_cast<const f32x4*>(a.pool + (slot * a.HV + hv) * (int64_t)plane + e);
  float* p = a.seg_state + ((int64_t)first * a.HV + hv) * plane + e;
  const float* d = a.seg_decay + (int64_t)first * a.HV + hv;
  const int64_t step = (int64_t)a.HV * plane;
  for (int i = 0; i < n; ++i, p += step, d += a.HV) {
    f32x4 mine = {0.f, 0.f, 0.f, 0.f};
    float f = 0.f;
    if (i + 1 < n) {
      mine = *reinterpret_cast<const f32x4*>(p);
      f = expf(*d);
    }
    *reinterpret_cast<f32x4*>(p) = s;
    s = s * f + mine;
  }
}

// Tokens of a segment: enough segments to fill the device, each long enough that the state it
// starts from and leaves is a small share of what it reads.
int segment_tokens(const SsmShape& s) {
  const int64_t blocks = cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock) * s.H;
  int64_t l = s.N * blocks / 1024;
  l = (l + 63) / 64 * 64;
  if (l < 512) l = 512;
  if (l > 8192) l = 8192;
  return s.N > l ? (int)l : 0;
}

// Segments of cut requests: each such request has more than lseg tokens, so at most twice
// N / lseg segments in all.
int64_t max_cut(const SsmShape& s, int lseg) { return lseg ? 2 * (s.N / lseg) : 0; }

struct ScanLayout {
  size_t state = 0, decay = 0, total = 0;
};
ScanLayout scan_layout(const SsmShape& s) {
  const int64_t n = max_cut(s, segment_tokens(s));
  ScanLayout L;
  L.decay = align256((size_t)n * s.HV * s.dv * s.dk * sizeof(float));
  L.total = L.decay + align256((size_t)n * s.HV * sizeof(float)) + 256;
  return L;
}

int64_t scan_blocks(const SsmShape& s) {
  const int lseg = segment_tokens(s);
  return (s.B + (lseg ? s.N / lseg : 0)) * s.H * cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock);
}

template <typename T, int DK, int CH>
hipError_t launch_scan(const SsmShape& s, const ScanArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)scan_blocks(s);
  if (a.lseg) {
    hipLaunchKernelGGL((ssm_scan_kernel<T, DK, CH, false>), dim3(blocks), dim3(kThreads), 0, st, a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int parts = s.dv * s.dk / 1024;
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)(s.B * s.HV * parts)), dim3(256), 0, st, a,
                       s.dv * s.dk, parts);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_scan_kernel<T, DK, CH, true>), dim3(blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t ssm_workspace(const SsmShape& s) { return scan_layout(s).total; }

bool ssm_prefill_grids_fit(const SsmShape& s) {
  return grid_ok(scan_blocks(s), kThreads) && grid_ok(s.B * s.HV * (s.dv * s.dk / 1024), 256);
}

hipError_t launch_ssm_prefill(const SsmShape& s, const void* C, const void* B, const void* x,
                              const float* dt, const float* A_log, const float* dt_bias,
                              const float* D, float* state, const int64_t* idx,
                              const int64_t* cu, void* out, char* ws, hipStream_t st) {
  const ScanLayout L = scan_layout(s);
  const int lseg = segment_tokens(s);
  ScanArgs a{C, B, x, dt, A_log, dt_bias, D, state, idx, cu, out, (float*)(ws + L.state),
             (float*)(ws + L.decay), s.N, s.B, s.pool, s.H, s.HV, s.dv, s.HV / s.H,
             (int)cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock), lseg,
             (int)max_cut(s, lseg)};
#define GDN_SCAN_CASE(DK, CHB)                                        \
  if (s.dk == DK)                                                     \
    return s.bf16 ? launch_scan<__bf16, DK, CHB>(s, a, st) : launch_scan<float, DK, 32>(s, a, st);
  GDN_SCAN_CASE(64, 64)
  GDN_SCAN_CASE(128, 64)
  GDN_SCAN_CASE(256, 32)
#undef GDN_SCAN_CASE
  return hipErrorInvalidValue;
}

}  // namespace layer
}  // namespace gdn
