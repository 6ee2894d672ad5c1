// C ABI of the layer operators (declared in include/gdn.h): host-side argument checks and
// launches of the short causal convolution, the selective state space scan and the gated norm.
#include "gdn.h"
#include "gdn_layer.h"

using namespace gdn::layer;

namespace {

bool dtype_ok(int32_t d) { return d == GDN_DTYPE_F32 || d == GDN_DTYPE_BF16; }

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Elements of a 16-byte vector.
int vec(bool bf16) { return bf16 ? 8 : 4; }

gdn_status_t check_conv(const gdn_conv_problem_t* p, ConvShape* s) {
  if (!p || p->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->batch < 0 || p->pool_size < 0) return GDN_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->dout_dtype)) return GDN_ERR_INVALID_ARG;
  if ((p->flags & ~GDN_CONV_SILU) != 0) return GDN_ERR_INVALID_ARG;
  if (p->channels[0] <= 0 || p->channels[1] < 0 || p->channels[2] < 0) return GDN_ERR_INVALID_ARG;
  const int64_t ch = (int64_t)p->channels[0] + p->channels[1] + p->channels[2];
  if (p->x_stride < ch) return GDN_ERR_INVALID_ARG;
  if (p->width < 1) return GDN_ERR_INVALID_ARG;
  if (p->width < 2 || p->width > 4) return GDN_ERR_UNSUPPORTED;
  // every offset of a tensor stays below 2^62
  if (ch > (1 << 24) || p->total_tokens > ((int64_t)1 << 31) || p->batch > ((int64_t)1 << 30) ||
      p->pool_size > ((int64_t)1 << 31) || p->x_stride > ((int64_t)1 << 28))
    return GDN_ERR_UNSUPPORTED;
  s->N = p->total_tokens;
  s->B = p->batch;
  s->pool = p->pool_size;
  s->x_stride = p->x_stride;
  s->dx_stride = p->dx_stride;
  s->ch = (int)ch;
  s->c1 = p->channels[0];
  s->c2 = p->channels[0] + p->channels[1];
  s->W = p->width;
  s->bf16 = p->dtype == GDN_DTYPE_BF16;
  s->dout_bf16 = p->dout_dtype == GDN_DTYPE_BF16;
  s->silu = (p->flags & GDN_CONV_SILU) != 0;
  // a vector of channels stays inside one output and starts on 16 bytes in every row
  const int v = vec(s->bf16);
  s->vec = s->c1 % v == 0 && s->c2 % v == 0 && s->ch % v == 0 && s->x_stride % v == 0;
  return GDN_OK;
}

gdn_status_t run_conv(const void* x, const float* weight, const float* bias, void* state,
                      const int64_t* idx, const int64_t* cu, void* out0, void* out1, void* out2,
                      const gdn_conv_problem_t* prob, bool decode, void* stream) {
  ConvShape s;
  const gdn_status_t ps = check_conv(prob, &s);
  if (ps != GDN_OK) return ps;
  if (decode && s.N != s.B) return GDN_ERR_INVALID_ARG;
  if (s.N == 0 || s.B == 0) return GDN_OK;
  if (!x || !weight || !out0 || (s.c2 > s.c1 && !out1) || (s.ch > s.c2 && !out2))
    return GDN_ERR_INVALID_ARG;
  if (decode ? !state : !cu) return GDN_ERR_INVALID_ARG;
  if (state && (!idx || s.pool < 1)) return GDN_ERR_INVALID_ARG;
  for (const void* p : {x, (const void*)weight, (const void*)bias, (const void*)state,
                        (const void*)out0, (const void*)out1, (const void*)out2})
    s.vec = s.vec && aligned16(p);
  if (!conv_grids_fit(s, false)) return GDN_ERR_UNSUPPORTED;
  void* const out[3] = {out0, out1, out2};
  const hipError_t e =
      decode ? launch_conv_decode(s, x, weight, bias, state, idx, out, (hipStream_t)stream)
             : launch_conv_fwd(s, x, weight, bias, state, idx, cu, out, (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status_t check_ssm(const gdn_problem_t* p, SsmShape* s) {
  if (!p) return GDN_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->batch < 0 || p->pool_size < 0) return GDN_ERR_INVALID_ARG;
  if (p->num_qk_heads <= 0 || p->num_v_heads <= 0 || p->num_v_heads % p->num_qk_heads != 0)
    return GDN_ERR_INVALID_ARG;
  if (p->head_k <= 0 || p->head_v <= 0 || !dtype_ok(p->qkv_dtype) || p->flags != 0)
    return GDN_ERR_INVALID_ARG;
  if (p->batch > 0 && p->pool_size < 1) return GDN_ERR_INVALID_ARG;
  for (const int32_t d : {p->head_k, p->head_v})
    if (d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
  if (p->num_v_heads > 65535 || p->batch > ((int64_t)1 << 30) ||
      p->pool_size > ((int64_t)1 << 31) || p->total_tokens > ((int64_t)1 << 30))
    return GDN_ERR_UNSUPPORTED;
  *s = SsmShape{p->total_tokens, p->batch,  p->pool_size, p->num_qk_heads,
                p->num_v_heads,  p->head_k, p->head_v,    p->qkv_dtype == GDN_DTYPE_BF16};
  return GDN_OK;
}

gdn_status_t check_norm(const gdn_norm_problem_t* p, bool gated, bool backward, NormShape* s) {
  if (!p || p->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (p->total_tokens < 0 || p->heads <= 0 || p->dim <= 0 || !dtype_ok(p->dtype))
    return GDN_ERR_INVALID_ARG;
  if ((p->flags & ~(GDN_NORM_RMS | GDN_NORM_GATE_FIRST)) != 0) return GDN_ERR_INVALID_ARG;
  if ((p->flags & GDN_NORM_GATE_FIRST) && !gated) return GDN_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f)) return GDN_ERR_INVALID_ARG;
  const int64_t row = (int64_t)p->heads * p->dim;
  if (p->x_stride < row || (gated && p->z_stride < row) ||
      (gated && backward && p->dz_stride < row))
    return GDN_ERR_INVALID_ARG;
  if (p->dim > 16384 || row > ((int64_t)1 << 28) || p->total_tokens > ((int64_t)1 << 31) ||
      p->x_stride > ((int64_t)1 << 30) || p->z_stride > ((int64_t)1 << 30) ||
      p->dz_stride > ((int64_t)1 << 30))
    return GDN_ERR_UNSUPPORTED;
  s->N = p->total_tokens;
  s->x_stride = p->x_stride;
  s->z_stride = p->z_stride;
  s->dz_stride = p->dz_stride;
  s->heads = p->heads;
  s->dim = p->dim;
  s->bf16 = p->dtype == GDN_DTYPE_BF16;
  s->rms = (p->flags & GDN_NORM_RMS) != 0;
  s->gate_first = (p->flags & GDN_NORM_GATE_FIRST) != 0;
  s->eps = p->eps;
  const int v = vec(s->bf16);
  s->vec = s->dim % v == 0 && s->x_stride % v == 0 && (!gated || s->z_stride % v == 0) &&
           (!gated || !backward || s->dz_stride % v == 0);
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_conv_fwd(const void* x, const float* weight, const float* bias, void* state_pool,
                          const int64_t* cache_indices, const int64_t* cu_seqlens, void* out0,
                          void* out1, void* out2, const gdn_conv_problem_t* prob, void* stream) {
  return run_conv(x, weight, bias, state_pool, cache_indices, cu_seqlens, out0, out1, out2, prob,
                  false, stream);
}

gdn_status_t gdn_conv_decode_fwd(const void* x, const float* weight, const float* bias,
                                 void* state_pool, const int64_t* cache_indices, void* out0,
                                 void* out1, void* out2, const gdn_conv_problem_t* prob,
                                 void* stream) {
  return run_conv(x, weight, bias, state_pool, cache_indices, nullptr, out0, out1, out2, prob,
                  true, stream);
}

size_t gdn_conv_bwd_workspace_size(const gdn_conv_problem_t* prob) {
  ConvShape s;
  return check_conv(prob, &s) == GDN_OK ? conv_bwd_workspace(s) : 0;
}

gdn_status_t gdn_conv_bwd(const void* x, const float* weight, const float* bias,
                          const void* state_pool, const int64_t* cache_indices,
                          const int64_t* cu_seqlens, const void* dout0, const void* dout1,
                          const void* dout2, const float* dstate, void* dx, float* dweight,
                          float* dbias, float* dstate0, const gdn_conv_problem_t* prob,
                          void* workspace, size_t workspace_bytes, void* stream) {
  ConvShape s;
  const gdn_status_t ps = check_conv(prob, &s);
  if (ps != GDN_OK) return ps;
  if (s.dx_stride < s.ch) return GDN_ERR_INVALID_ARG;
  if (s.dx_stride > ((int64_t)1 << 28)) return GDN_ERR_UNSUPPORTED;
  if (!weight || !dweight || (bias != nullptr) != (dbias != nullptr)) return GDN_ERR_INVALID_ARG;
  if (s.B > 0 && (!cu_seqlens || (state_pool && (!cache_indices || s.pool < 1))))
    return GDN_ERR_INVALID_ARG;
  if (s.N > 0 && s.B > 0 &&
      (!x || !dx || !dout0 || (s.c2 > s.c1 && !dout1) || (s.ch > s.c2 && !dout2)))
    return GDN_ERR_INVALID_ARG;
  s.vec = s.vec && s.dx_stride % vec(s.bf16) == 0;
  for (const void* p : {x, (const void*)weight, (const void*)bias, state_pool, dout0, dout1,
                        dout2, (const void*)dstate, (const void*)dx})
    s.vec = s.vec && aligned16(p);
  if (s.B == 0) s.N = 0;  // every row is padding
  const size_t need = conv_bwd_workspace(s);
  if (!conv_grids_fit(s, true)) return GDN_ERR_UNSUPPORTED;
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255) != 0))
    return GDN_ERR_WORKSPACE;
  const void* const dout[3] = {dout0, dout1, dout2};
  const hipError_t e =
      launch_conv_bwd(s, x, weight, bias, state_pool, cache_indices, cu_seqlens, dout, dstate, dx,
                      dweight, dbias, s.B > 0 ? dstate0 : nullptr, (float*)workspace,
                      (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_ssm_workspace_size(const gdn_problem_t* prob) {
  SsmShape s;
  return check_ssm(prob, &s) == GDN_OK ? ssm_workspace(s) : 0;
}

gdn_status_t gdn_ssm_prefill_fwd(const void* C, const void* B, const void* x, const float* dt,
                                 const float* A_log, const float* dt_bias, const float* D,
                                 float* state_pool, const int64_t* cache_indices,
                                 const int64_t* cu_seqlens, void* out, const gdn_problem_t* prob,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  SsmShape s;
  const gdn_status_t ps = check_ssm(prob, &s);
  if (ps != GDN_OK) return ps;
  if (s.N == 0 || s.B == 0) return GDN_OK;
  if (!C || !B || !x || !dt || !A_log || !dt_bias || !state_pool || !cache_indices ||
      !cu_seqlens || !out)
    return GDN_ERR_INVALID_ARG;
  for (const void* p : {C, B, x, (const void*)out, (const void*)state_pool})
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!ssm_prefill_grids_fit(s)) return GDN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < ssm_workspace(s) || ((uintptr_t)workspace & 255) != 0)
    return GDN_ERR_WORKSPACE;
  const hipError_t e = launch_ssm_prefill(s, C, B, x, dt, A_log, dt_bias, D, state_pool,
                                          cache_indices, cu_seqlens, out, (char*)workspace,
                                          (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status_t gdn_ssm_decode_fwd(const void* C, const void* B, const void* x, const float* dt,
                                const float* A_log, const float* dt_bias, const float* D,
                                float* state_pool, const int64_t* cache_indices, void* out,
                                const gdn_problem_t* prob, void* stream) {
  SsmShape s;
  const gdn_status_t ps = check_ssm(prob, &s);
  if (ps != GDN_OK) return ps;
  if (s.N != s.B) return GDN_ERR_INVALID_ARG;  // exactly one token per request
  if (s.B == 0) return GDN_OK;
  if (!C || !B || !x || !dt || !A_log || !dt_bias || !state_pool || !cache_indices || !out)
    return GDN_ERR_INVALID_ARG;
  for (const void* p : {C, B, x, (const void*)out, (const void*)state_pool})
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!ssm_token_grid_fits(s)) return GDN_ERR_UNSUPPORTED;
  const hipError_t e = launch_ssm_decode(s, C, B, x, dt, A_log, dt_bias, D, state_pool,
                                         cache_indices, out, (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

gdn_status_t gdn_norm_fwd(const void* x, const float* weight, const float* bias, const void* z,
                          void* out, const gdn_norm_problem_t* prob, void* stream) {
  NormShape s;
  const gdn_status_t ps = check_norm(prob, z != nullptr, false, &s);
  if (ps != GDN_OK) return ps;
  if (s.N == 0) return GDN_OK;
  if (!x || !weight || !out) return GDN_ERR_INVALID_ARG;
  for (const void* p : {x, (const void*)weight, (const void*)bias, z, (const void*)out})
    s.vec = s.vec && aligned16(p);
  const hipError_t e = launch_norm_fwd(s, x, weight, bias, z, out, (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

size_t gdn_norm_bwd_workspace_size(const gdn_norm_problem_t* prob) {
  NormShape s;
  // the strides of z and dz play no part in the size
  return check_norm(prob, prob && prob->z_stride > 0, false, &s) == GDN_OK ? norm_bwd_workspace(s)
                                                                           : 0;
}

gdn_status_t gdn_norm_bwd(const void* x, const float* weight, const float* bias, const void* z,
                          const void* dout, void* dx, void* dz, float* dweight, float* dbias,
                          const gdn_norm_problem_t* prob, void* workspace, size_t workspace_bytes,
                          void* stream) {
  NormShape s;
  const gdn_status_t ps = check_norm(prob, z != nullptr, true, &s);
  if (ps != GDN_OK) return ps;
  if (!weight || !dweight || (bias != nullptr) != (dbias != nullptr)) return GDN_ERR_INVALID_ARG;
  if (s.N > 0 && (!x || !dout || !dx || (z != nullptr) != (dz != nullptr)))
    return GDN_ERR_INVALID_ARG;
  for (const void* p : {x, (const void*)weight, (const void*)bias, z, dout, (const void*)dx,
                        (const void*)dz})
    s.vec = s.vec && aligned16(p);
  const size_t need = norm_bwd_workspace(s);
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255) != 0))
    return GDN_ERR_WORKSPACE;
  const hipError_t e = launch_norm_bwd(s, x, weight, bias, z, dout, dx, dz, dweight, dbias,
                                       (float*)workspace, (hipStream_t)stream);
  return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
}

}  // extern "C"
