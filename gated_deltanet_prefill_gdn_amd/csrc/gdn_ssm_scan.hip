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
// Requests longer than a segment are cut into equal pieces: a first launch forms each piece's
// state from zero, a second joins the pieces' states in order into their start states and the
// final one, and a third forms the outputs of all pieces side by side, and takes the requests that
// are not cut from start to end. Only the scalar decay per head lies between two pieces, so the
// join is one multiply-add per state entry and piece. A piece's state is summed from its end, and
// only as far back as weights are not zero in fp32: heads that forget fast stop after a few chunks,
// so long pieces are taken in parts, which spread the slow heads over the device.
//
// Precision: bf16 inputs enter the products as they are. The decayed x of the state's update are
// three bf16 (24 bits), since states are fp32 results. What only outputs take, which end as bf16, is
// two bf16 (16 bits): the decayed scores, the state that S C reads, and the decayed x where a piece's
// state is only formed to be read so. One bf16 each would be a rounding as large as the output's own
// (errors of 1.79e-3 of the outputs' size instead of 1.66e-3, twelve times a rounding where terms
// cancel; the two cases below took 982 and 362 us a call with it). For fp32 inputs every operand is three bf16 and
// a product takes the six pairs of parts that reach 2^-24: 2.7 times the rate of the fp32 matrix
// instructions. Gates are fp32, the sums that differences are taken of fixed point or fp64, and
// exponents are only taken of differences that are not positive, so strong decays underflow to zero
// and nothing overflows.
//
// Measured, bf16, calls back to back: 131072 tokens, 32 heads of 128 x 128, 1164 us (outputs 919, 3.9
// TB/s of what they move); 8 ragged requests of 33860 tokens, 64 heads of 64 x 128 that share C and B
// by eights, 425 us (outputs 307). No unit is full in the outputs: the matrix cores are busy 36 and
// 24 % of the time, the vector units 46 and 38, LDS 42 and 31. Two waves a SIMD and two or three
// barriers a chunk leave waits open, and behind the longest piece of the ragged requests a fifth of
// the device idles.
#include <type_traits>

#include "gdn_layer_chunk.h"

namespace gdn {
namespace layer {
namespace {

using mfma::kperm;
using mfma::mma_bf16;

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kColsWave = 32, kColsBlock = kColsWave * kWaves;  // value columns

struct ScanArgs {
  const void *C, *B, *x;
  const float *dt, *A_log, *dt_bias, *D;
  float* pool;
  const int64_t *idx, *cu;
  void* out;
  float* seg_state;   // [segments of cut requests][parts][HV][dv][dk]: the parts' states, then in
                      // the first part's place the segment's start state
  float* seg_decay;   // [segments of cut requests][parts][HV]: sum of g from a part's start to the
                      // segment's end, kNoState where the part's state is zero and not written
  int64_t N, nreq, npool;
  int H, HV, dv, rep, blocks_per_group;
  int lseg;           // tokens of a segment (a multiple of 64), 0: nothing is cut
  int max_cut;        // places in seg_state
  int parts;          // of a segment, whose states are formed side by side
  int short_len;      // requests of at most this many tokens are left to the token kernel
};

constexpr float kNoState = 1.f;  // (sums of g are not positive)

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

// Segment number `seg` of the call, by a scan over the requests, 64 at a time in every wave.
__device__ __forceinline__ bool find_segment(const ScanArgs& a, int seg, Segment& s) {
  const int lane = threadIdx.x & 63;
  int len;
  if (a.lseg == 0) {
    s.req = seg;
    s.index = 0;
    s.count = 1;
    s.ws = 0;
    len = 0;
  } else {
    int before = 0, before_cut = 0;
    bool found = false;
    for (int64_t base = 0; base < a.nreq; base += 64) {
      const int64_t b = base + lane;
      int mine = 0;
      const int n = b < a.nreq ? pieces_of(end_of(a, b) - begin_of(a, b), a.lseg, mine) : 0;
      const int inc = wave_inclusive(n), cut = wave_inclusive(n > 1 ? n : 0);
      const uint64_t over = __ballot(before + inc > seg);
      if (over) {
        const int k = __builtin_ctzll(over);
        s.count = __builtin_amdgcn_readlane(n, k);
        s.index = seg - before - (__builtin_amdgcn_readlane(inc, k) - s.count);
        s.ws = before_cut + __builtin_amdgcn_readlane(cut, k) - s.count + s.index;
        s.req = base + k;
        len = __builtin_amdgcn_readlane(mine, k);
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(inc, 63);
      before_cut += __builtin_amdgcn_readlane(cut, 63);
    }
    if (!found) return false;
  }
  const int64_t begin = begin_of(a, s.req), end = end_of(a, s.req);
  s.t0 = begin + (int64_t)s.index * len;
  s.t1 = s.index + 1 < s.count ? s.t0 + len : end;
  const int64_t slot = a.idx[s.req];
  if (s.count > 1 && s.ws >= a.max_cut) return false;  // cu_seqlens breaks its precondition
  return s.t0 < s.t1 && end - begin > a.short_len && slot >= 0 && slot < a.npool;
}

constexpr float kLog2e = 1.44269504088896340736f;

// x, or lo where it is below that. (NaN stays NaN.)
__device__ __forceinline__ float above(float x, float lo) { return x < lo ? lo : x; }

// log(1 + e^x) = max(x, 0) + log1p(z), z = e^-|x|: with w = 1 + z rounded, log1p(z) is
// log(w) z / (w - 1), in which the rounding of w cancels, and z where w is 1.
__device__ __forceinline__ float softplusf(float x) {
  const float z = exp2_(-fabsf(x) * kLog2e), w = 1.f + z;
  const float l = __builtin_amdgcn_logf(w) * (z * __builtin_amdgcn_rcpf((w - 1.f) * kLog2e));
  return fmaxf(x, 0.f) + (w == 1.f ? z : l);
}

// v from another lane of the same row of 16, chosen by a DPP control code; 0 from outside it.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 b = __builtin_bit_cast(i32x2, v);
  return __builtin_bit_cast(double, i32x2{dpp<CTRL>(b[0]), dpp<CTRL>(b[1])});
}
// Sum over this lane and those before it in its row of 16 lanes.
template <typename R>
__device__ __forceinline__ R row_prefix(R v) {
  v += dpp<0x111>(v);  // from 1, 2, 4, 8 lanes before
  v += dpp<0x112>(v);
  v += dpp<0x114>(v);
  v += dpp<0x118>(v);
  return v;
}
// Sum over the lanes behind this one in its row.
__device__ __forceinline__ float row_behind(float v) {
  v = dpp<0x101>(v);  // from 1, 2, 4, 8 lanes behind
  v += dpp<0x101>(v);
  v += dpp<0x102>(v);
  v += dpp<0x104>(v);
  v += dpp<0x108>(v);
  return v;
}
__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ double lane_of(double v, int lane) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 b = __builtin_bit_cast(i32x2, v);
  return __builtin_bit_cast(double, i32x2{__builtin_amdgcn_readlane(b[0], lane),
                                          __builtin_amdgcn_readlane(b[1], lane)});
}

// The gates of one head in one chunk, an entry per token.
// Outputs take e to differences of running sums of g (to base 2, as every g here), which go into the
// thousands where some tokens erase a state that those between them keep: fp32 sums would leave
// errors of up to 2^-10 there. fp32 inputs: the sum from the chunk's start in fp64. bf16 inputs: from
// the tile's start in steps of 2^-19 (2^-16 off over a tile at most), whose differences are exact.
template <int CH, typename R>
struct Gates {
  R G[CH];
  float step[CH];      // d
  float eG[CH];        // e^G
  float row[CH];       // e^{G_t - G at the start of t's tile}
  float w[CH];         // d e^{G_n - G}: weight in the state's update
  // d_j e^{G at tile k's start - G_j} for the tokens j before it, k = 1, 2, ..: 16 k from at(k) on
  float col[CH / 16 * (CH / 16 - 1) / 2 * 16];
  static __device__ __forceinline__ int at(int k) { return 8 * k * (k - 1); }
  float total[4];              // G_n (its own 16 bytes)
};

// Staging of a tile of CH rows x COLS entries: 16-byte pieces in registers between the load and
// the LDS store, so that the next chunk's rows travel while this one is worked on.
template <typename T, int CH, int COLS>
struct Stage {
  static constexpr int V = 16 / (int)sizeof(T);
  static constexpr int PER_ROW = COLS / V, PIECES = CH * PER_ROW / kThreads;
  static constexpr int ROWS = kThreads / PER_ROW;  // rows of one piece of all threads
  static_assert(CH * PER_ROW % kThreads == 0 && kThreads % PER_ROW == 0, "whole rows at a time");
  u32x4 r[PIECES];
  __device__ __forceinline__ void load(const T* base, int64_t ld, int rows, int cols) {
    const int ldb = (int)(ld * (int)sizeof(T));
    const rsrc_t q = chunk_rows(base, ldb, rows, cols * (int)sizeof(T));
    const int at = (int)(threadIdx.x / PER_ROW) * ldb + (int)(threadIdx.x % PER_ROW) * 16;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      r[i] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(q, at + i * ROWS * ldb, 0, 0));
  }
  // as NP tiles of bf16 parts, `plane` entries apart
  template <int NP, bool WIDE>
  __device__ __forceinline__ void store(__bf16* to, int plane, int ld) const {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int p = i * kThreads + threadIdx.x, row = p / PER_ROW, c = p % PER_ROW * V;
      if constexpr (NP == 1) {
        if constexpr (WIDE) {
          *reinterpret_cast<u32x4*>(to + row * ld + c) = r[i];
        } else {  // rows start on 8 bytes
          u32x2* const q = reinterpret_cast<u32x2*>(to + row * ld + c);
          q[0] = u32x2{r[i][0], r[i][1]};
          q[1] = u32x2{r[i][2], r[i][3]};
        }
      } else {
        const f32x4 v = __builtin_bit_cast(f32x4, r[i]);
        uint32_t lo[NP], hi[NP];
        split<NP, true>(v[0], v[1], lo);
        split<NP, true>(v[2], v[3], hi);
#pragma unroll
        for (int p = 0; p < NP; ++p)
          *reinterpret_cast<u32x2*>(to + p * plane + row * ld + c) = u32x2{lo[p], hi[p]};
      }
    }
  }
};

// The tiles of the lower triangle of CH / 16 x CH / 16 tiles, dealt to the waves so that most of a
// wave's tiles are of one row: three in rows 3 and 2, (1, 0), (1, 1) and (3, 3), (0, 0); of 32
// tokens (0, 0), (1, 0) and (1, 1).
template <int NT>
__device__ __forceinline__ bool deal(int wave, int i, int& tt, int& jt) {
  if constexpr (NT == 4) {
    tt = 3 - wave;
    jt = i;
    if (wave == 2 && i == 2) tt = jt = 3;
    return wave < 3 || i == 0;
  } else {
    tt = wave > 0;
    jt = wave > 1;
    return wave < 3;
  }
}

// What a workgroup does with its segment: a whole request, outputs and state; the state of a
// piece from zero; the outputs of a piece from its start state.
enum Mode { kWhole, kState, kOutput };

// HEADS: heads of a workgroup at most, two where a head has 64 columns.
template <typename T, int DK, int CH, int HEADS>
struct Dims {
  static constexpr int NP = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of an input
  static constexpr int PS = sizeof(T) == 4 ? 3 : 2;  // ... of the decayed scores and of S in S C
  // LDS rows. C is read in 8-byte pieces down 16 rows: 4.5 cycles for a wave's read where the
  // stride is 2 mod 4 words, 8 or 16 elsewhere. B and x are read transposed and in 16-byte pieces:
  // no conflicts and 4.9 cycles where it is 8 mod 16 words, 8 elsewhere (measured).
  static constexpr int LDC = DK + 12, LDB = DK + 16, LDX = kColsBlock + 16, LDP = CH + 8;
  static constexpr int TileC = CH * LDC, TileB = CH * LDB, TileX = CH * LDX, TileP = CH * LDP;
  using R = typename std::conditional<sizeof(T) == 4, double, int>::type;
  using G = Gates<CH, R>;
  // LDS: B, x, four gate sets; with outputs also C and the heads' decayed scores. For bf16 inputs
  // those of two heads start in C's place, which has been read by then: two workgroups a CU have
  // 80 KB each.
  static constexpr bool Over = sizeof(T) == 2 && HEADS == 2;
  static constexpr int AtX = NP * TileB * 2, AtG = AtX + NP * TileX * 2;
  static constexpr int AtC = AtG + kWaves * (int)sizeof(G), EndC = AtC + NP * TileC * 2;
  static constexpr int AtP = Over ? AtC : EndC, EndP = AtP + HEADS * PS * TileP * 2;
  static constexpr int Bytes = EndP > EndC ? EndP : EndC;
  static_assert(AtX % 16 == 0 && AtG % 16 == 0 && AtC % 16 == 0 && AtP % 16 == 0, "16-byte rows");
};

// A piece's state: sg is the part of the piece, `ws` its place and `end` the piece's end.
template <typename T, int DK, int CH, int HEADS, Mode MODE>
__device__ __forceinline__ void scan_segment(const ScanArgs& a, const Segment& sg, int in_seg,
                                             char* lds, int64_t ws = 0, int64_t end = 0) {
  using D = Dims<T, DK, CH, HEADS>;
  using R = typename D::R;
  using G = typename D::G;
  constexpr bool F32 = sizeof(T) == 4, OUT = MODE != kState;
  constexpr int NP = D::NP, PS = D::PS;
  // ... of the update's decayed x: the state of a piece's outputs is only read by S C
  constexpr int NU = MODE == kOutput ? PS : 3;
  constexpr int NT = CH / 16, NK = CH / 32;      // token tiles, k steps over tokens
  constexpr int NS = DK / 16, NKS = DK / 32;     // state tiles, k steps over state entries
  constexpr int TRI = NT == 4 ? 3 : 1;           // tiles of scores for a wave at most
  constexpr int LDC = D::LDC, LDB = D::LDB, LDX = D::LDX, LDP = D::LDP;
  constexpr int kTileC = D::TileC, kTileB = D::TileB, kTileX = D::TileX, kTileP = D::TileP;
  __bf16* const s_b = reinterpret_cast<__bf16*>(lds);
  __bf16* const s_x = reinterpret_cast<__bf16*>(lds + D::AtX);
  G* const s_g = reinterpret_cast<G*>(lds + D::AtG);
  __bf16* const s_c = reinterpret_cast<__bf16*>(lds + D::AtC);

  const int h = in_seg / a.blocks_per_group;
  const int col0 = in_seg % a.blocks_per_group * kColsBlock;  // of the group's columns
  const int vc = a.rep * a.dv;
  const int ncols = vc - col0 < kColsBlock ? vc - col0 : kColsBlock;

  const int tid = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  int lane = tid & 63, r = lane & 15, g = lane >> 4;
  const bool live = kColsWave * wv < ncols;
  const int wcol = live ? col0 + kColsWave * wv : col0;
  const int hv = h * a.rep + wcol / a.dv, p0 = wcol % a.dv;
  const int64_t slot = a.idx[sg.req];
  // Heads of the workgroup, and the one this wave's columns belong to. The four gate sets hold
  // four chunks of one head or two of two: each wave forms one set, of head gh and the chunk
  // gc after the batch's first.
  const int hv0 = h * a.rep + col0 / a.dv, nh = HEADS == 1 ? 1 : (ncols + a.dv - 1) / a.dv;
  const int batch = nh == 2 ? 2 : 4, gh = nh == 2 ? wv >> 1 : 0, gc = nh == 2 ? wv & 1 : wv;
  const int hw = nh == 2 ? kColsWave * wv / a.dv : 0;
  // decayed scores, row t; entry 32 k + 8 g + e is token j = 32 k + kperm(g, e)
  __bf16* const s_p = reinterpret_cast<__bf16*>(lds + D::AtP);
  auto gate_set = [&](int head, int chunk) -> G& {
    return s_g[nh == 2 ? 2 * head + (chunk & 1) : chunk & 3];
  };

  const T* const gB = reinterpret_cast<const T*>(a.B) + (int64_t)h * DK;
  const T* const gC = reinterpret_cast<const T*>(a.C) + (int64_t)h * DK;
  const T* const gx = reinterpret_cast<const T*>(a.x) + (int64_t)h * vc + col0;
  T* const gout = reinterpret_cast<T*>(a.out) + (int64_t)hv * a.dv + p0;
  const int64_t ldb = (int64_t)a.H * DK, ldx = (int64_t)a.HV * a.dv;

  // S^T: st[s tile][column tile], entries 16 s + 4 g .. + 3 of column p0 + 16 pt + r
  acc4 st[NS][2];
  const float* from = nullptr;
  const int64_t plane = (int64_t)a.dv * DK;
  if (OUT) {
    from = MODE == kOutput ? a.seg_state + ((int64_t)sg.ws * a.parts * a.HV + hv) * plane
                        : a.pool + (slot * a.HV + hv) * plane;
    from += (int64_t)(p0 + r) * DK + 4 * g;
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
      st[s][pt] = OUT && live ? *reinterpret_cast<const acc4*>(from + 16 * pt * DK + 16 * s)
                              : acc4{0.f, 0.f, 0.f, 0.f};

  const float decay = above(-expf(a.A_log[hv0 + gh]) * kLog2e, -3e38f), dtb = a.dt_bias[hv0 + gh];
  const float dskip = a.D ? a.D[hv] : 0.f;
  // a piece's state: sum of g from the chunks walked to the piece's end, of each head
  float behind[HEADS] = {};
  if constexpr (MODE == kState) {
    float* const s_sum = reinterpret_cast<float*>(lds);
    bool more = sg.t0 < sg.t1;
    for (int64_t t = sg.t1; more && t < end; t += 4 * kThreads) {
      float sum[HEADS] = {};
#pragma unroll
      for (int hh = 0; hh < HEADS; ++hh) {
        if (hh >= nh) break;
        const float rate = above(-expf(a.A_log[hv0 + hh]) * kLog2e, -3e38f);
        const float shift = a.dt_bias[hv0 + hh];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int64_t k = t + u * kThreads + tid;
          if (k < end) sum[hh] += rate * softplusf(a.dt[k * a.HV + hv0 + hh] + shift);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) sum[hh] += __shfl_xor(sum[hh], off, 64);
        if (lane == 0) s_sum[hh * kWaves + wv] = sum[hh];
      }
      __syncthreads();
      more = false;
#pragma unroll
      for (int hh = 0; hh < HEADS; ++hh)
        if (hh < nh) {
#pragma unroll
          for (int k = 0; k < kWaves; ++k) behind[hh] += s_sum[hh * kWaves + k];
          more = more || !(exp2_(behind[hh]) == 0.f);
        }
      __syncthreads();
    }
    if (!more) {  // no token, or every weight is zero in fp32
      if (live && p0 == 0 && lane == 0) a.seg_decay[ws * a.HV + hv] = kNoState;
      return;
    }
  }

  Stage<T, CH, DK> qb, qc;  // the next chunk's rows (two chunks ahead are no faster)
  Stage<T, CH, kColsBlock> qx;
  float qdt = 0.f;
  auto fetch = [&](int64_t t) {
    const int rows = sg.t1 - t < CH ? (int)(sg.t1 - t) : CH;
    qb.load(gB + t * ldb, ldb, rows, DK);
    if constexpr (OUT) qc.load(gC + t * ldb, ldb, rows, DK);
    qx.load(gx + t * ldx, ldx, rows, ncols);
  };
  // The chunks in the order of the walk: outputs from the front. A piece's state alone is summed
  // from its end, where the weights of its chunks are known, and the walk stops at chunks that
  // have none.
  const int chunks = (int)((sg.t1 - sg.t0 + CH - 1) / CH);
  auto place = [&](int n) { return sg.t0 + (int64_t)(OUT ? n : chunks - 1 - n) * CH; };
  auto fetch_dt = [&](int n) {  // of this wave's set in the batch of chunks from the n-th on
    qdt = 0.f;
    if (n + gc < chunks) {
      const int64_t t = place(n + gc), left = sg.t1 - t;
      qdt = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(
                     chunk_rows(a.dt + t * a.HV + hv0 + gh, (int64_t)a.HV * 4,
                                left < CH ? (int)left : CH, 4),
                     lane * a.HV * 4, 0, 0));
    }
  };
  fetch(place(0));
  fetch_dt(0);

  for (int chunk = 0; chunk < chunks; ++chunk) {
    const int64_t t0 = place(chunk);
    if constexpr (MODE == kWhole || (MODE == kOutput && HEADS == 2)) {
      // Places in LDS are formed anew for every chunk: kept in registers they spill, and a
      // reload waits for the next chunk's rows, which were asked for before it (8 ragged requests
      // with two heads a workgroup 477 us, so 418).
      asm volatile("" : "+v"(lane));
      r = lane & 15;
      g = lane >> 4;
    }
    if (chunk > 0) __syncthreads();  // the chunk before has been read
    const int rows = sg.t1 - t0 < CH ? (int)(sg.t1 - t0) : CH;
    qb.template store<NP, true>(s_b, kTileB, LDB);
    if constexpr (OUT) qc.template store<NP, false>(s_c, kTileC, LDC);
    qx.template store<NP, true>(s_x, kTileX, LDX);
    if (chunk % batch == 0) {
      // a gate set, a lane per token; rows past the end have no step and no decay
      G& gt = gate_set(gh, chunk + gc);
      const bool in = lane < CH && chunk + gc < chunks && place(chunk + gc) + lane < sg.t1;
      const float step = in ? softplusf(qdt + dtb) : 0.f;
      // (a g of -1e30 decays to zero as any lower one does, and sums of them stay finite)
      const float gl = in ? above(decay * step, -1e30f) : 0.f;
      using S = typename std::conditional<F32, double, float>::type;
      const S local = row_prefix((S)gl);
      S at[NT + 1];  // G before each tile, and at the end
      at[0] = 0;
#pragma unroll
      for (int k = 0; k < NT; ++k) at[k + 1] = at[k] + lane_of(local, 16 * k + 15);
      S mine = at[0];
#pragma unroll
      for (int k = 1; k < NT; ++k) mine = lane >= 16 * k ? at[k] : mine;
      const S Gp = mine + local;
      const float behind_me = row_behind(gl);  // of g in this lane's tile
      float tiles = 0.f;  // of g in the tiles behind this lane's, up to tile k
#pragma unroll
      for (int k = 1; k < NT; ++k) {
        if constexpr (OUT)
          if (lane < 16 * k)
            gt.col[G::at(k) + lane] =
                step * exp2_(F32 ? (float)(at[k] - Gp) : behind_me + tiles);
        tiles += lane < 16 * k ? (float)lane_of(local, 16 * k + 15) : 0.f;
      }
      if (lane < CH) {
        if constexpr (OUT) {
          // (what is below 2^-160 is zero, and sixteen of it fit)
          if constexpr (F32)
            gt.G[lane] = Gp;
          else
            gt.G[lane] = row_prefix((int)__builtin_rintf(fmaxf(gl, -160.f) * 0x1p19f));
          gt.step[lane] = step;
          gt.eG[lane] = exp2_((float)Gp);
          gt.row[lane] = exp2_((float)local);
        }
        gt.w[lane] = step * exp2_(behind_me + tiles);
      }
      if (lane == 0) gt.total[0] = (float)at[NT];
      fetch_dt(chunk + batch);
    }
    __syncthreads();
    if (chunk + 1 < chunks) fetch(place(chunk + 1));
    const G& gt = gate_set(hw, chunk);

    acc4 y[NT][2];  // Y^T: columns 16 pt + 4 g .. + 3 of token 16 t + r
    acc4 sc[TRI];   // scores^T, j x t: each wave some of the tiles
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < TRI; ++i) {
        int tt, jt;
        if (!deal<NT>(wv, i, tt, jt)) break;
        acc4 half[2] = {acc4{0.f, 0.f, 0.f, 0.f}, acc4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < NKS; ++k)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const u32x2* const cp = reinterpret_cast<const u32x2*>(
                s_c + p * kTileC + (16 * tt + r) * LDC + 32 * k + 8 * g);
            const bfrag c = bfrag_of(cp[0], cp[1]);
#pragma unroll
            for (int q = 0; q + p < NP; ++q)
              half[k % 2] =
                  mma_bf16(*reinterpret_cast<const bfrag*>(s_b + q * kTileB +
                                                           (16 * jt + r) * LDB + 32 * k + 8 * g),
                           c, half[k % 2]);
          }
        sc[i] = half[0] + half[1];
      }
      // the scores, decayed for each of the workgroup's heads
      auto decay_scores = [&]() {
#pragma unroll
        for (int i = 0; i < TRI; ++i) {
          int tt, jt;
          if (!deal<NT>(wv, i, tt, jt)) break;
          for (int hh = 0; hh < HEADS; ++hh) {
            if (hh >= nh) break;
            const G& gs = gate_set(hh, chunk);
            __bf16* const to = s_p + hh * PS * kTileP + (16 * tt + r) * LDP + 32 * (jt / 2) + 8 * g +
                               4 * (jt % 2);
            float v[4];
            if (jt < tt) {
              const acc4 c = *reinterpret_cast<const acc4*>(&gs.col[G::at(tt) + 16 * jt + 4 * g]);
              const float row = gs.row[16 * tt + r];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = sc[i][e] * (c[e] * row);
            } else {
              const acc4 d = *reinterpret_cast<const acc4*>(&gs.step[16 * jt + 4 * g]);
              const R Gt = gs.G[16 * tt + r];
              R Gj[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) Gj[e] = gs.G[16 * jt + 4 * g + e];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float lag = (float)(Gt - Gj[e]) * (F32 ? 1.f : 0x1p-19f);
                float ex = sc[i][e] * (exp2_(lag) * d[e]);
                asm volatile("" : "+v"(ex));  // no branch around each entry
                v[e] = 4 * g + e <= r ? ex : 0.f;
              }
              if (jt % 2 == 0)  // the tile beside it shares its k step
#pragma unroll
                for (int p = 0; p < PS; ++p)
                  *reinterpret_cast<u32x2*>(to + p * kTileP + 4) = u32x2{0, 0};
            }
            uint32_t lo[PS], hi[PS];
            split<PS, F32>(v[0], v[1], lo);
            split<PS, F32>(v[2], v[3], hi);
#pragma unroll
            for (int p = 0; p < PS; ++p)
              *reinterpret_cast<u32x2*>(to + p * kTileP) = u32x2{lo[p], hi[p]};
          }
        }
      };
      if constexpr (!D::Over) decay_scores();
      // S C, and its decay
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) y[t][pt] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NKS; ++k) {
        bfrag cf[NT][NP];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < NP; ++p)
            cf[t][p] = frag_kperm(s_c + p * kTileC + (16 * t + r) * LDC + 32 * k, g);
        // (reads left among the products wait one by one: 131072 tokens 930 us instead of 894)
        if constexpr (!F32) __builtin_amdgcn_sched_barrier(0);
        bfrag sb[PS][2];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          u32x4 words[PS];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            uint32_t part[PS];
            const acc4 v = st[2 * k + e / 4][pt];
            split<PS, F32>(v[e % 4], v[e % 4 + 1], part);
#pragma unroll
            for (int p = 0; p < PS; ++p) words[p][e / 2] = part[p];
          }
#pragma unroll
          for (int p = 0; p < PS; ++p) sb[p][pt] = bf16x8_from_u32x4(words[p]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bfrag c = cf[t][p];
#pragma unroll
            for (int q = 0; q + p < PS; ++q)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) y[t][pt] = mma_bf16(sb[q][pt], c, y[t][pt]);
          }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float e = gt.eG[16 * t + r];
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) y[t][pt] *= e;
      }
      if constexpr (D::Over) {
        __syncthreads();  // C has been read
        decay_scores();
      }
      __syncthreads();
    }
    bfrag xf[NP][2][NK];  // x, column p0 + 16 pt + r, tokens 32 k + kperm
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int pt = 0; pt < 2; ++pt)
#pragma unroll
        for (int k = 0; k < NK; ++k)
          xf[p][pt][k] = frag_col(s_x + p * kTileX, LDX, kColsWave * wv + 16 * pt, k, g, r);

    if constexpr (OUT) {
      // + scores times x
      const rsrc_t qo = chunk_rows(gout + t0 * ldx, ldx * (int)sizeof(T), live ? rows : 1,
                                   live ? kColsWave * (int)sizeof(T) : 0);
      const __bf16* const ph = s_p + hw * PS * kTileP;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc4 yp[2];  // fp32 keeps the two sums apart: fewer roundings at the size of the output
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) yp[pt] = F32 ? acc4{0.f, 0.f, 0.f, 0.f} : y[t][pt];
#pragma unroll
        for (int k = 0; k <= t / 2; ++k)
#pragma unroll
          for (int q = 0; q < PS; ++q) {
            const bfrag pf = *reinterpret_cast<const bfrag*>(ph + q * kTileP + (16 * t + r) * LDP +
                                                             32 * k + 8 * g);
#pragma unroll
            for (int p = 0; p < NP && p + q < PS; ++p)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) yp[pt] = mma_bf16(xf[p][pt][k], pf, yp[pt]);
          }
        // + D x, and out: four columns of one token per lane
        const int row = 16 * t + r;
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          const int at = row * LDX + kColsWave * wv + 16 * pt + 4 * g;
          float xv[4], o[4];
#pragma unroll
          for (int p = NP - 1; p >= 0; --p) {
            const bf16x4 xp = *reinterpret_cast<const bf16x4*>(s_x + p * kTileX + at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              xv[i] = p == NP - 1 ? (float)xp[i] : xv[i] + (float)xp[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i] = __builtin_fmaf(dskip, xv[i], yp[pt][i]);
            if constexpr (F32) o[i] += y[t][pt][i];
          }
          const int to = row * (int)(ldx * sizeof(T)) + (16 * pt + 4 * g) * (int)sizeof(T);
          if constexpr (F32) {
            __builtin_amdgcn_raw_buffer_store_b128(
                __builtin_bit_cast(u32x4, f32x4{o[0], o[1], o[2], o[3]}), qo, to, 0, 0);
          } else {
            __builtin_amdgcn_raw_buffer_store_b64(
                __builtin_bit_cast(u32x2, bf16x4{(__bf16)o[0], (__bf16)o[1], (__bf16)o[2],
                                                 (__bf16)o[3]}),
                qo, to, 0, 0);
          }
        }
      }
    }

    // S^T <- e^{G_n} S^T + B^T (w x)
    if (MODE == kOutput && chunk + 1 == chunks) break;  // nobody reads this state
    // outputs: the state before decays over the chunk; a piece's state: the chunk's part decays
    // over those behind it
    const float eGn = OUT ? exp2_(gt.total[0]) : exp2_(behind[hw]);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      u32x4 xw[NU][2];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i] = gt.w[32 * k + kperm(g, e + i)];
          if constexpr (!OUT) w[i] *= eGn;
        }
#pragma unroll
        for (int pt = 0; pt < 2; ++pt) {
          float v[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            v[i] = (float)xf[NP - 1][pt][k][e + i];
#pragma unroll
            for (int p = NP - 2; p >= 0; --p) v[i] += (float)xf[p][pt][k][e + i];
          }
          uint32_t part[NU];
          split<NU, F32>(v[0] * w[0], v[1] * w[1], part);
#pragma unroll
          for (int p = 0; p < NU; ++p) xw[p][pt][e / 2] = part[p];
        }
      }
#pragma unroll
      for (int s = 0; s < NS; s += 2) {  // two tiles: four sums between two products of one
        if constexpr (OUT)
          if (k == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt) st[s + i][pt] *= eGn;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          bfrag b[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) b[i] = frag_col(s_b + p * kTileB, LDB, 16 * (s + i), k, g, r);
#pragma unroll
          for (int q = 0; q + p < NU; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int pt = 0; pt < 2; ++pt)
                st[s + i][pt] = mma_bf16(b[i], bf16x8_from_u32x4(xw[q][pt]), st[s + i][pt]);
        }
      }
    }
    if constexpr (!OUT) {
      bool more = false;
#pragma unroll
      for (int hh = 0; hh < HEADS; ++hh)
        if (hh < nh) {
          behind[hh] += gate_set(hh, chunk).total[0];
          more = more || !(exp2_(behind[hh]) == 0.f);
        }
      if (!more) break;  // every earlier weight is zero in fp32, and so is the piece's decay
    }
  }

  if (!live || MODE == kOutput) return;
  float* to = MODE == kWhole ? a.pool + (slot * a.HV + hv) * plane
                             : a.seg_state + (ws * a.HV + hv) * plane;
  to += (int64_t)(p0 + r) * DK + 4 * g;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int pt = 0; pt < 2; ++pt)
      *reinterpret_cast<acc4*>(to + 16 * pt * DK + 16 * s) = st[s][pt];
  if (MODE == kState && p0 == 0 && lane == 0) a.seg_decay[ws * a.HV + hv] = behind[hw];
}

// The pieces' states (OUTPUT false); the outputs of pieces, and whole requests.
// Workgroups of a CU that the registers are held to (fp32: LDS for one at dk >= 128): outputs
// keep the next C, the scores and the states' parts in them too, states alone leave room for three
// (8 ragged requests, 64 heads of 64 x 128: 412 us a call, with two 425). At dk = 256 a compiler left
// free takes more than half the registers, and one workgroup a CU: 16384 tokens, 8 heads of 256 x
// 256, 230 us instead of 179, 10 ragged requests 451 instead of 324.
template <typename T, int DK, bool OUTPUT>
constexpr int kGroupsPerCU = sizeof(T) == 4 ? 1 : OUTPUT || DK == 256 ? 2 : 3;
template <typename T, int DK, int CH, int HEADS, bool OUTPUT>
__global__ __launch_bounds__(kThreads, (kGroupsPerCU<T, DK, OUTPUT>)) void ssm_scan_kernel(
    ScanArgs a) {
  using D = Dims<T, DK, CH, HEADS>;
  __shared__ __align__(16) char lds[OUTPUT ? D::Bytes : D::AtC];
  // Workgroups are dealt to the eight XCDs in turn: the column blocks of a (segment, group) go to
  // one of them, one after the other, and find B and C in its L2. The XCD of a group changes from
  // segment to segment, since groups differ in how far a piece's state reaches back.
  const int turn = blockIdx.x / 8, row = turn / a.blocks_per_group;
  const int unit = row * 8 + (blockIdx.x + 3 * row + row / 8) % 8;
  const int in_seg = unit % a.H * a.blocks_per_group + turn % a.blocks_per_group;
  const int parts = OUTPUT ? 1 : a.parts, seg = unit / a.H / parts;
  if (a.lseg == 0 && seg >= a.nreq) return;  // units are a multiple of eight
  Segment sg;
  if (!find_segment(a, seg, sg)) return;
  if constexpr (OUTPUT) {
    if (sg.count > 1)
      scan_segment<T, DK, CH, HEADS, kOutput>(a, sg, in_seg, lds);
    else
      scan_segment<T, DK, CH, HEADS, kWhole>(a, sg, in_seg, lds);
  } else if (sg.count > 1) {
    const int part = unit / a.H % parts;
    const int len = ((int)(sg.t1 - sg.t0) + 64 * parts - 1) / (64 * parts) * 64;
    const int64_t end = sg.t1;
    sg.t0 += (int64_t)part * len;
    sg.t1 = sg.t0 + len < end ? sg.t0 + len : end;
    scan_segment<T, DK, CH, HEADS, kState>(a, sg, in_seg, lds, (int64_t)sg.ws * parts + part, end);
  }
}

// Start states of a cut request's pieces, in place of the pieces' own states, and its final state.
template <int PARTS>
__global__ __launch_bounds__(256) void ssm_join_kernel(ScanArgs a, int plane, int parts) {
  const int part = blockIdx.x % parts;  // every parts-th run of 1024 entries from this one on
  const int64_t pair = blockIdx.x / parts;
  const int64_t req = pair / a.HV;
  const int hv = (int)(pair - req * a.HV);
  const int64_t slot = a.idx[req];
  int len;
  const int n = pieces_of(end_of(a, req) - begin_of(a, req), a.lseg, len);
  if (n <= 1 || slot < 0 || slot >= a.npool) return;
  int first = 0;  // place of the request's first segment
  for (int64_t base = 0; base < req; base += 64) {
    const int64_t b = base + (threadIdx.x & 63);
    const int k = b < req ? pieces_of(end_of(a, b) - begin_of(a, b), a.lseg, len) : 0;
    first += __builtin_amdgcn_readlane(wave_inclusive(k > 1 ? k : 0), 63);
  }
  if (first + n > a.max_cut) return;  // cu_seqlens breaks its precondition
  constexpr int AHEAD = 8 / PARTS;  // pieces whose states are in flight together
  const int64_t step = (int64_t)a.HV * plane;
  for (int e = (part * 256 + threadIdx.x) * 4; e < plane; e += parts * 1024) {
    f32x4* const home = reinterpret_cast<f32x4*>(a.pool + (slot * a.HV + hv) * (int64_t)plane + e);
    const float* d = a.seg_decay + (int64_t)first * PARTS * a.HV + hv;
    float* p = a.seg_state + ((int64_t)first * PARTS * a.HV + hv) * plane + e;
    f32x4 s = *home;
    for (int i = 0; i < n; i += AHEAD, p += AHEAD * PARTS * step, d += AHEAD * PARTS * a.HV) {
      float G[AHEAD][PARTS];
      f32x4 mine[AHEAD][PARTS];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int j = 0; j < PARTS; ++j)
          G[u][j] = i + u < n ? d[(u * PARTS + j) * a.HV] : kNoState;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int j = 0; j < PARTS; ++j) {
          mine[u][j] = f32x4{0.f, 0.f, 0.f, 0.f};
          if (!(G[u][j] > 0.f))
            mine[u][j] = *reinterpret_cast<const f32x4*>(p + (u * PARTS + j) * step);
        }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        if (i + u >= n) break;
        *reinterpret_cast<f32x4*>(p + u * PARTS * step) = s;
        s *= G[u][0] > 0.f ? 0.f : exp2_(G[u][0]);
#pragma unroll
        for (int j = 0; j < PARTS; ++j) s += mine[u][j];
      }
    }
    *home = s;
  }
}

// Tokens of a piece at most (lseg 0: no request is cut). A workgroup's time goes with its tokens,
// and `slots` of them run at a time, so pieces are sized to fill k rounds of the device, with
// half a piece more for every request, k = 1 .. 4: more rounds even out pieces of different
// lengths, fewer spare the joins, which cost what kPieceTokens tokens do (a piece's state is
// written, joined and read: 256 KB at dk = 128 for 128 columns, whose tokens take 0.75 KB; with
// 350 instead of 1000, 8 ragged requests of 33860 tokens in all, 64 heads of 64 x 128, take 432
// us instead of 412, and 16 requests of 1024 are cut for nothing, 231 us instead of 155).
// Requests that fill the device by their number alone (from 4096 / blocks of them on) are not cut:
// equal ones need not be, but a long one among them is walked by one workgroup a column block. A
// prompt of 32768 tokens beside 125 single tokens, heads as above, takes 2.85 ms, alone 0.37 ms.
// A piece's state in one part, two or four, by its length: one request of 131072 tokens, 32 heads
// of 128 x 128 (pieces of 8512), 1144, 1106 and 1081 us a call; the 8 ragged requests (of 2880) 428,
// 411 and 421; 16384 tokens, 8 heads of 256 x 256 (of 576), 178, 198 and 227.
constexpr int kPieceTokens = 1000;
struct Cut {
  int lseg, parts;
};
Cut cut_of(const SsmShape& s) {
  const int64_t blocks = cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock) * s.H;
  constexpr int64_t slots = 512;
  int64_t best = 0, cost = INT64_MAX;
  for (int k = 1; k <= 4; ++k) {
    const int64_t pieces2 = 2 * k * slots / blocks - s.B;  // twice the pieces for N tokens
    if (pieces2 <= 0) continue;
    const int64_t l = cdiv(cdiv(2 * s.N, pieces2), 64) * 64;
    if (k * (l + kPieceTokens) < cost) {
      cost = k * (l + kPieceTokens);
      best = l;
    }
  }
  if (best < 512) best = best == 0 ? 0 : 512;
  if (best == 0 || s.N <= best) return Cut{0, 1};
  return Cut{(int)best, best < 2048 ? 1 : best < 4096 ? 2 : 4};
}

// Requests of at most this many tokens run token by token, where the mean length says that most
// are and there are enough to fill the device (a call that splits pays a launch for the longer
// ones too): 512 requests of 4 tokens, 32 heads of 128 x 128, take 392 us there and 438 in chunks,
// of 8 tokens 570 and 445.
int short_tokens(const SsmShape& s) {
  return s.N <= 4 * s.B && s.B * s.HV * (s.dv / 64) >= 2048 ? 4 : 0;
}

// Segments of cut requests: one of L tokens has at most L / lseg + 1, and each has more than lseg
// tokens, so that there are at most min(B, N / lseg) of them.
int64_t max_cut(const SsmShape& s, int lseg) {
  if (!lseg) return 0;
  const int64_t full = s.N / lseg;
  return full + (s.B < full ? s.B : full);
}

struct ScanLayout {
  size_t state = 0, decay = 0, total = 0;
};
ScanLayout scan_layout(const SsmShape& s) {
  const Cut c = cut_of(s);
  const int64_t n = max_cut(s, c.lseg) * c.parts;
  ScanLayout L;
  L.decay = align256((size_t)n * s.HV * s.dv * s.dk * sizeof(float));
  L.total = L.decay + align256((size_t)n * s.HV * sizeof(float)) + 256;
  return L;
}

int64_t scan_blocks(const SsmShape& s, int parts) {
  const int lseg = cut_of(s).lseg;
  return cdiv((s.B + (lseg ? s.N / lseg : 0)) * parts * s.H, 8) * 8 *
         cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock);
}

// Workgroups of a state in the join: enough to fill the device, few where many requests are likely
// not cut.
int join_parts(const SsmShape& s) {
  int parts = s.dv * s.dk / 1024;
  while (parts > 1 && s.B * s.HV * (parts / 2) >= 2048) parts /= 2;
  return parts;
}

template <typename T, int DK, int CH, int HEADS>
hipError_t launch_scan(const SsmShape& s, const ScanArgs& a, hipStream_t st) {
  if (a.lseg) {
    hipLaunchKernelGGL((ssm_scan_kernel<T, DK, CH, HEADS, false>),
                       dim3((unsigned)scan_blocks(s, a.parts)), dim3(kThreads), 0, st, a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int parts = join_parts(s);
    const auto join = a.parts == 1   ? ssm_join_kernel<1>
                      : a.parts == 2 ? ssm_join_kernel<2>
                                     : ssm_join_kernel<4>;
    hipLaunchKernelGGL(join, dim3((unsigned)(s.B * s.HV * parts)), dim3(256), 0, st, a,
                       s.dv * s.dk, parts);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_scan_kernel<T, DK, CH, HEADS, true>), dim3((unsigned)scan_blocks(s, 1)),
                     dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t ssm_workspace(const SsmShape& s) { return scan_layout(s).total; }

bool ssm_prefill_grids_fit(const SsmShape& s) {
  // the byte offsets inside a chunk's rows are 32-bit
  const int64_t row = (s.HV * (int64_t)s.dv > s.H * (int64_t)s.dk ? s.HV * (int64_t)s.dv
                                                                  : s.H * (int64_t)s.dk) * 4;
  return row * 64 <= 0x7FFFFFFF && grid_ok(scan_blocks(s, cut_of(s).parts), kThreads) &&
         (!short_tokens(s) || ssm_token_grid_fits(s)) &&
         (!cut_of(s).lseg || grid_ok(s.B * s.HV * join_parts(s), 256));
}

hipError_t launch_ssm_prefill(const SsmShape& s, const void* C, const void* B, const void* x,
                              const float* dt, const float* A_log, const float* dt_bias,
                              const float* D, float* state, const int64_t* idx,
                              const int64_t* cu, void* out, char* ws, hipStream_t st) {
  const ScanLayout L = scan_layout(s);
  const Cut c = cut_of(s);
  ScanArgs a{C, B, x, dt, A_log, dt_bias, D, state, idx, cu, out, (float*)(ws + L.state),
             (float*)(ws + L.decay), s.N, s.B, s.pool, s.H, s.HV, s.dv, s.HV / s.H,
             (int)cdiv((int64_t)(s.HV / s.H) * s.dv, kColsBlock), c.lseg,
             (int)max_cut(s, c.lseg), c.parts, short_tokens(s)};
  if (a.short_len)
    if (const hipError_t e = launch_ssm_short(s, C, B, x, dt, A_log, dt_bias, D, state, idx, cu,
                                              out, a.short_len, st);
        e != hipSuccess)
      return e;
#define GDN_SCAN_CASE(DK, CHB)                                          \
  if (s.dk == DK) {                                                     \
    if (s.bf16)                                                         \
      return s.dv == 64 ? launch_scan<__bf16, DK, CHB, 2>(s, a, st)     \
                        : launch_scan<__bf16, DK, CHB, 1>(s, a, st);    \
    return s.dv == 64 ? launch_scan<float, DK, 32, 2>(s, a, st)         \
                      : launch_scan<float, DK, 32, 1>(s, a, st);        \
  }
  GDN_SCAN_CASE(64, 64)
  GDN_SCAN_CASE(128, 64)
  GDN_SCAN_CASE(256, 32)
#undef GDN_SCAN_CASE
  return hipErrorInvalidValue;
}

}  // namespace layer
}  // namespace gdn
