// C ABI of the selective state space block (declared in include/rapt.h): convolution, scan, layer norm.
// Validation, workspace sizing and dispatch, as in api.cu.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/rapt.h"
#include "kernels.h"

namespace {

using rapt::DType;

constexpr long long kMostRows = 1LL << 30;  // tokens of a call: room for a tile past the last in 31 bits

bool off(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool any_off16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (off(p, 16)) return true;
  return false;
}
bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return true;
  return false;
}
bool among(const void* out, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (out != nullptr && out == p) return true;
  return false;
}
bool known_dtype(int t) { return t == RAPT_F32 || t == RAPT_BF16; }
bool known_act(rapt_act a) { return a >= RAPT_ACT_NONE && a <= RAPT_ACT_SIGMOID; }
DType to_dt(int t) { return t == RAPT_F32 ? DType::F32 : DType::BF16; }
rapt_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RAPT_OK : RAPT_ERR_CUDA; }
cudaStream_t as_stream(rapt_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

rapt::Docs dense_docs(int32_t B, int32_t L, uint32_t* dev_status) {
  return {nullptr, dev_status, B, L, B * L, L};
}

// ---------------------------------------------------------------- convolution
rapt_status check_conv(rapt_dtype dtype, int32_t D, int32_t W, rapt_act act, int64_t x_stride, long long docs) {
  if (!known_dtype(dtype) || !known_act(act)) return RAPT_ERR_UNSUPPORTED;
  if (D < 1 || D > 1 << 24 || docs < 1 || docs * D > 1LL << 38) return RAPT_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return RAPT_ERR_UNSUPPORTED;
  return x_stride < D || x_stride > 1LL << 40 ? RAPT_ERR_INVALID_ARG : RAPT_OK;
}

rapt_status conv(const rapt::Docs& docs, const void* x, int64_t x_stride, rapt_dtype dtype, int32_t D,
                 const float* w, const float* bias, int32_t W, rapt_act act, const void* state, void* out,
                 void* state_final, rapt_stream_t stream) {
  if (w == nullptr || (docs.total_rows > 0 && (x == nullptr || out == nullptr))) return RAPT_ERR_INVALID_ARG;
  if (any_off16({x, w, bias, state, out, state_final}) || off(docs.dev_status, 4)) return RAPT_ERR_INVALID_ARG;
  if (among(out, {x, state, w, bias, state_final}) || among(state_final, {x, state, w, bias}))
    return RAPT_ERR_INVALID_ARG;
  rapt::ConvArgs a{};
  a.docs = docs;
  a.x = x; a.x_stride = static_cast<long>(x_stride);
  a.w = w; a.bias = bias;
  a.state = state; a.out = out; a.state_final = state_final;
  a.D = D; a.W = W; a.act = static_cast<rapt::Act>(act);
  return from_cuda(rapt::launch_conv(to_dt(dtype), a, as_stream(stream)));
}

// ---------------------------------------------------------------- scan
// Sizes and types of a scan's inputs; its pointers are checked where there are tokens.
rapt_status check_shape(const rapt_ssm_inputs* in) {
  if (in == nullptr) return RAPT_ERR_INVALID_ARG;
  const auto size = [](int v) { return v == 16 || v == 32 || v == 64 || v == 128; };
  if (!known_dtype(in->dtype) || !size(in->P) || !size(in->Ns)) return RAPT_ERR_UNSUPPORTED;
  if (in->H < 1 || in->G < 1 || in->H % in->G != 0 || in->H > 1 << 20) return RAPT_ERR_INVALID_ARG;
  return RAPT_OK;
}
rapt_status check_inputs(const rapt_ssm_inputs* in, long long rows, long long docs, const void* out) {
  if (rows > kMostRows || docs < 1 || docs * in->H >= (1LL << 31) / 64) return RAPT_ERR_INVALID_ARG;
  if (any_null({in->A}) || any_off16({in->A, in->D, in->dt_bias})) return RAPT_ERR_INVALID_ARG;
  if (rows == 0) return RAPT_OK;
  if (any_null({in->x, in->dt, in->B, in->C, out})) return RAPT_ERR_INVALID_ARG;
  const int64_t e = in->dtype == RAPT_F32 ? 4 : 2;
  if (any_off16({in->x, in->B, in->C, in->z, out}) || off(in->dt, e)) return RAPT_ERR_INVALID_ARG;
  const int64_t wide = static_cast<int64_t>(in->H) * in->P, narrow = static_cast<int64_t>(in->G) * in->Ns;
  const auto bad = [e](int64_t stride, int64_t least) {
    return stride < least || stride > 1LL << 37 || stride * e % 16 != 0;  // (a tensor map's stride is below 2^40 bytes)
  };
  if (bad(in->x_stride, wide) || bad(in->B_stride, narrow) || bad(in->C_stride, narrow) ||
      (in->z != nullptr && bad(in->z_stride, wide)) || in->dt_stride < in->H || in->dt_stride > 1LL << 37)
    return RAPT_ERR_INVALID_ARG;
  return among(out, {in->x, in->dt, in->B, in->C, in->z}) ? RAPT_ERR_INVALID_ARG : RAPT_OK;
}

rapt::SsmArgs make_args(const rapt_ssm_inputs* in, const rapt::Docs& docs, bool packed) {
  rapt::SsmArgs a{};
  a.docs = docs;
  a.x = in->x; a.dt = in->dt; a.B = in->B; a.C = in->C; a.z = in->z;
  a.xs = in->x_stride; a.dts = in->dt_stride; a.bs = in->B_stride; a.cs = in->C_stride; a.zs = in->z_stride;
  a.A = in->A; a.D = in->D; a.dt_bias = in->dt_bias;
  a.H = in->H; a.P = in->P; a.G = in->G; a.N = in->Ns;
  a.softplus = in->dt_softplus != 0;
  a.packed = packed;
  return a;
}

bool on_tensor_cores(const rapt_ssm_inputs* in) { return rapt::ssm_tc_supported(to_dt(in->dtype), in->P, in->Ns); }

rapt::SsmPlan plan(const rapt_ssm_inputs* in, const rapt::SsmArgs& a) {
  return on_tensor_cores(in) ? rapt::ssm_plan_tc(a) : rapt::ssm_plan_simt(a);
}

rapt_status scan(const rapt_ssm_inputs* in, const rapt::Docs& docs, const float* S0, void* out, float* S_final,
                 void* workspace, size_t workspace_bytes, rapt_stream_t stream) {
  if (any_off16({S0, S_final}) || off(docs.dev_status, 4)) return RAPT_ERR_INVALID_ARG;
  if (among(S_final, {S0, in->x, in->dt, in->B, in->C, in->z, out, in->A, in->D, in->dt_bias}) || among(out, {S0}))
    return RAPT_ERR_INVALID_ARG;
  rapt::SsmArgs a = make_args(in, docs, docs.cu_seqlens != nullptr);
  const rapt::SsmPlan p = plan(in, a);
  if (workspace_bytes < p.ws_bytes || (p.ws_bytes > 0 && (workspace == nullptr || off(workspace, 16))))
    return RAPT_ERR_WORKSPACE;
  a.S0 = S0; a.S_final = S_final; a.out = out;
  a.ws = static_cast<float*>(workspace);
  a.nseg = p.nseg; a.seg_len = p.seg_len; a.sorted = p.sorted;
  return from_cuda(on_tensor_cores(in) ? rapt::launch_ssm_tc(a, as_stream(stream))
                                       : rapt::launch_ssm_simt(to_dt(in->dtype), a, as_stream(stream)));
}

rapt_status check_norm(rapt_dtype dtype, int32_t T, int32_t D, float eps) {
  if (!known_dtype(dtype)) return RAPT_ERR_UNSUPPORTED;
  // the root's instruction takes a subnormal for zero: a row of equal values would become NaN
  if (T < 0 || D < 1 || !std::isfinite(eps) || !(eps >= FLT_MIN)) return RAPT_ERR_INVALID_ARG;
  return D > rapt::kResidualNormMaxD ? RAPT_ERR_UNSUPPORTED : RAPT_OK;
}

}  // namespace

extern "C" {

rapt_status rapt_conv_prefill_fwd(const void* x, int64_t x_stride, rapt_dtype dtype, int32_t B, int32_t L,
                                  int32_t D, const float* w, const float* bias, int32_t W, rapt_act act,
                                  const void* state, void* out, void* state_final, rapt_stream_t stream) {
  const rapt_status st = check_conv(dtype, D, W, act, x_stride, B);
  if (st != RAPT_OK) return st;
  if (L < 0 || static_cast<long long>(B) * L > kMostRows) return RAPT_ERR_INVALID_ARG;
  return conv(dense_docs(B, L, nullptr), x, x_stride, dtype, D, w, bias, W, act, state, out, state_final, stream);
}

rapt_status rapt_conv_varlen_fwd(const void* x, int64_t x_stride, rapt_dtype dtype, int32_t T, int32_t D,
                                 const int32_t* cu_seqlens, int32_t N, const float* w, const float* bias,
                                 int32_t W, rapt_act act, const void* state, void* out, void* state_final,
                                 uint32_t* dev_status, rapt_stream_t stream) {
  const rapt_status st = check_conv(dtype, D, W, act, x_stride, N);
  if (st != RAPT_OK) return st;
  if (T < 0 || T > kMostRows || cu_seqlens == nullptr || off(cu_seqlens, 4)) return RAPT_ERR_INVALID_ARG;
  const rapt::Docs docs{cu_seqlens, dev_status, N, 0, T, INT_MAX};
  return conv(docs, x, x_stride, dtype, D, w, bias, W, act, state, out, state_final, stream);
}

rapt_status rapt_conv_decode_step(const void* x, int64_t x_stride, rapt_dtype dtype, int32_t N, int32_t D,
                                  const float* w, const float* bias, int32_t W, rapt_act act, void* state,
                                  void* out, rapt_stream_t stream) {
  const rapt_status st = check_conv(dtype, D, W, act, x_stride, N);
  if (st != RAPT_OK) return st;
  if (any_null({x, w, state, out}) || any_off16({x, w, bias, state, out})) return RAPT_ERR_INVALID_ARG;
  if (among(out, {x, w, bias, state}) || among(state, {x, w, bias})) return RAPT_ERR_INVALID_ARG;
  return from_cuda(rapt::launch_conv_step(to_dt(dtype), x, static_cast<long>(x_stride), w, bias, state, out, N, D, W,
                                          static_cast<rapt::Act>(act), as_stream(stream)));
}

size_t rapt_ssm_prefill_workspace_size(const rapt_ssm_inputs* in, int32_t B, int32_t L) {
  if (check_shape(in) != RAPT_OK || B < 1 || L < 0 || static_cast<long long>(B) * L > kMostRows) return 0;
  return plan(in, make_args(in, dense_docs(B, L, nullptr), false)).ws_bytes;
}

rapt_status rapt_ssm_prefill_fwd(const rapt_ssm_inputs* in, int32_t B, int32_t L, const float* S0, void* out,
                                 float* S_final, uint32_t* dev_status, void* workspace, size_t workspace_bytes,
                                 rapt_stream_t stream) {
  rapt_status st = check_shape(in);
  if (st != RAPT_OK) return st;
  if (B < 1 || L < 0) return RAPT_ERR_INVALID_ARG;
  st = check_inputs(in, static_cast<long long>(B) * L, B, out);
  if (st != RAPT_OK) return st;
  if (L == 0 && S_final == nullptr) return RAPT_OK;
  return scan(in, dense_docs(B, L, dev_status), S0, out, S_final, workspace, workspace_bytes, stream);
}

size_t rapt_ssm_varlen_workspace_size(const rapt_ssm_inputs* in, int32_t T, int32_t N, int32_t max_seqlen) {
  if (check_shape(in) != RAPT_OK || T < 0 || T > kMostRows || N < 1 || max_seqlen < 0) return 0;
  return plan(in, make_args(in, {nullptr, nullptr, N, 0, T, max_seqlen < T ? max_seqlen : T}, true)).ws_bytes;
}

rapt_status rapt_ssm_varlen_fwd(const rapt_ssm_inputs* in, int32_t T, const int32_t* cu_seqlens, int32_t N,
                                int32_t max_seqlen, const float* S0, void* out, float* S_final,
                                uint32_t* dev_status, void* workspace, size_t workspace_bytes,
                                rapt_stream_t stream) {
  rapt_status st = check_shape(in);
  if (st != RAPT_OK) return st;
  if (T < 0 || N < 1 || max_seqlen < 0 || cu_seqlens == nullptr || off(cu_seqlens, 4)) return RAPT_ERR_INVALID_ARG;
  st = check_inputs(in, T, N, out);
  if (st != RAPT_OK) return st;
  const rapt::Docs docs{cu_seqlens, dev_status, N, 0, T, max_seqlen < T ? max_seqlen : T};
  return scan(in, docs, S0, out, S_final, workspace, workspace_bytes, stream);
}

rapt_status rapt_ssm_decode_step(const rapt_ssm_inputs* in, int32_t N, float* S, void* out, rapt_stream_t stream) {
  rapt_status st = check_shape(in);
  if (st != RAPT_OK) return st;
  if (N < 1) return RAPT_ERR_INVALID_ARG;
  st = check_inputs(in, N, N, out);
  if (st != RAPT_OK) return st;
  if (S == nullptr || off(S, 16) || among(S, {in->x, in->dt, in->B, in->C, in->z, out, in->A, in->D, in->dt_bias}))
    return RAPT_ERR_INVALID_ARG;
  rapt::SsmArgs a = make_args(in, dense_docs(N, 1, nullptr), false);
  a.out = out;
  return from_cuda(rapt::launch_ssm_step(to_dt(in->dtype), a, S, as_stream(stream)));
}

rapt_status rapt_layer_norm_fwd(const void* x, rapt_dtype dtype, int32_t T, int32_t D, const float* w,
                                const float* b, float eps, void* y, rapt_stream_t stream) {
  const rapt_status st = check_norm(dtype, T, D, eps);
  if (st != RAPT_OK) return st;
  if (T == 0) return RAPT_OK;
  if (any_null({x, y}) || any_off16({x, w, b, y}) || among(y, {w, b})) return RAPT_ERR_INVALID_ARG;
  rapt::LayerNormArgs a{};
  a.x = x; a.w = w; a.b = b; a.out = y;
  a.T = T; a.D = D; a.eps = eps;
  return from_cuda(rapt::launch_layer_norm_fwd(to_dt(dtype), a, as_stream(stream)));
}

size_t rapt_layer_norm_bwd_workspace_size(int32_t T, int32_t D, rapt_dtype dtype) {
  return check_norm(dtype, T, D, 1.f) != RAPT_OK ? 0 : rapt::layer_norm_ws_bytes(T, D, to_dt(dtype));
}

rapt_status rapt_layer_norm_bwd(const void* dy, const void* x, rapt_dtype dtype, int32_t T, int32_t D,
                                const float* w, float eps, void* dx, float* dw, float* db, void* workspace,
                                size_t workspace_bytes, rapt_stream_t stream) {
  const rapt_status st = check_norm(dtype, T, D, eps);
  if (st != RAPT_OK) return st;
  if (T > 0 && any_null({dy, x})) return RAPT_ERR_INVALID_ARG;  // an empty [T, D] tensor has no address
  if (any_off16({dy, x, w, dx, dw, db})) return RAPT_ERR_INVALID_ARG;
  if (among(dx, {w, dw, db}) || among(dw, {x, dy, w, db}) || among(db, {x, dy, w})) return RAPT_ERR_INVALID_ARG;
  const bool sums = dw != nullptr || db != nullptr;
  const size_t need = sums ? rapt::layer_norm_ws_bytes(T, D, to_dt(dtype)) : 0;
  if (workspace_bytes < need || (need > 0 && (workspace == nullptr || off(workspace, 16)))) return RAPT_ERR_WORKSPACE;
  rapt::LayerNormArgs a{};
  a.x = x; a.dy = dy; a.w = w; a.out = dx;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.T = T; a.D = D; a.eps = eps;
  return from_cuda(rapt::launch_layer_norm_bwd(to_dt(dtype), a, dw, db, as_stream(stream)));
}

}  // extern "C"
