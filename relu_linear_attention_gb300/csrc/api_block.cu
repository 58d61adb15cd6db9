// C ABI of the operators around the attention (declared in include/rapt.h): residual norms, gated
// feed-forward, gradients of projections. Validation, workspace sizing and dispatch, as in api.cu.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/rapt.h"
#include "kernels.h"

namespace {

using rapt::DType;

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool any_off16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (off16(p)) return true;
  return false;
}
bool known_act(rapt_act a) { return a >= RAPT_ACT_NONE && a <= RAPT_ACT_SIGMOID; }
rapt::Act to_act(rapt_act a) { return static_cast<rapt::Act>(a); }
DType to_dt(rapt_dtype t) { return t == RAPT_F32 ? DType::F32 : DType::BF16; }
rapt_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RAPT_OK : RAPT_ERR_CUDA; }
cudaStream_t as_stream(rapt_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Whether two of the given pointers (nulls aside) are the same.
bool any_same(std::initializer_list<const void*> ps) {
  for (auto a = ps.begin(); a != ps.end(); ++a)
    for (auto b = a + 1; b != ps.end(); ++b)
      if (*a != nullptr && *a == *b) return true;
  return false;
}
// Whether an output is an input's pointer.
bool aliases(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (const void* o : outs)
    for (const void* i : ins)
      if (o != nullptr && o == i) return true;
  return false;
}
bool bad_status_word(const uint32_t* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

rapt_status check_norm(rapt_dtype dtype, int32_t T, int32_t D, rapt_act act, float eps) {
  if ((dtype != RAPT_F32 && dtype != RAPT_BF16) || !known_act(act)) return RAPT_ERR_UNSUPPORTED;
  // the root's instruction takes a subnormal for zero: a row of zeros would become NaN
  if (T < 0 || D < 1 || !std::isfinite(eps) || !(eps >= FLT_MIN)) return RAPT_ERR_INVALID_ARG;
  if (D > rapt::kResidualNormMaxD) return RAPT_ERR_UNSUPPORTED;
  return RAPT_OK;
}

// M x N x K of a product in tiles: positive, rows of whole 16 bytes, a count of tiles that leaves room
// for the parts of a split sum in 31 bits, and no tile whose sum takes longer than the kernel's waits (a
// 64-deep slice of it takes 0.27 us: 2^26 are 0.3 s of 1 s).
rapt_status check_gemm(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N < 1 || K < 1) return RAPT_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0) return RAPT_ERR_UNSUPPORTED;
  if (M > 1 << 26 || N > 1 << 24 || K > 1 << 24) return RAPT_ERR_INVALID_ARG;
  const long long most = 1LL << 38;  // 2^24 tiles of 128 x 128
  if (static_cast<long long>(M) * N > most || static_cast<long long>(M) * K > most ||
      static_cast<long long>(N) * K > most)
    return RAPT_ERR_INVALID_ARG;
  return RAPT_OK;
}

rapt_status zero_bf16(void* p, long long n, rapt_stream_t stream) {
  return p == nullptr ? RAPT_OK : from_cuda(cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 2, as_stream(stream)));
}

}  // namespace

extern "C" {

rapt_status rapt_residual_norm_fwd(const void* x, const void* y, const void* gate, rapt_dtype dtype,
                                   int32_t T, int32_t D, rapt_act act, const float* w_post,
                                   const float* scale, const float* w_pre, float eps, void* r, void* h,
                                   rapt_stream_t stream) {
  const rapt_status st = check_norm(dtype, T, D, act, eps);
  if (st != RAPT_OK) return st;
  if (T == 0) return RAPT_OK;
  if ((r == nullptr && h == nullptr) || (h != nullptr && w_pre == nullptr)) return RAPT_ERR_INVALID_ARG;
  if (y == nullptr && (gate != nullptr || w_post != nullptr || scale != nullptr)) return RAPT_ERR_INVALID_ARG;
  if (x == nullptr) return RAPT_ERR_INVALID_ARG;
  if (any_off16({x, y, gate, w_post, scale, w_pre, r, h})) return RAPT_ERR_INVALID_ARG;
  if (any_same({r, h})) return RAPT_ERR_INVALID_ARG;
  rapt::ResidualNormArgs a{};
  a.x = x; a.y = y; a.gate = gate;
  a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
  a.r = r; a.h = h;
  a.T = T; a.D = D; a.act = to_act(act); a.eps = eps;
  return from_cuda(rapt::launch_residual_norm_fwd(to_dt(dtype), a, as_stream(stream)));
}

size_t rapt_residual_norm_bwd_workspace_size(int32_t T, int32_t D, rapt_dtype dtype) {
  if (check_norm(dtype, T, D, RAPT_ACT_NONE, 1.f) != RAPT_OK) return 0;
  return rapt::residual_norm_ws_bytes(T, D, to_dt(dtype));
}

rapt_status rapt_residual_norm_bwd(const void* dr, const void* dh, const void* x, const void* y,
                                   const void* gate, rapt_dtype dtype, int32_t T, int32_t D,
                                   rapt_act act, const float* w_post, const float* scale,
                                   const float* w_pre, float eps, void* dx, void* dy, void* dgate,
                                   float* dw_post, float* dscale, float* dw_pre, void* workspace,
                                   size_t workspace_bytes, rapt_stream_t stream) {
  const rapt_status st = check_norm(dtype, T, D, act, eps);
  if (st != RAPT_OK) return st;
  if ((dw_post != nullptr && w_post == nullptr) || (dscale != nullptr && scale == nullptr) ||
      (dw_pre != nullptr && w_pre == nullptr))
    return RAPT_ERR_INVALID_ARG;
  if (T > 0) {  // an empty [T, D] tensor has no address
    if (dr == nullptr && dh == nullptr) return RAPT_ERR_INVALID_ARG;
    if (dh != nullptr && (x == nullptr || w_pre == nullptr)) return RAPT_ERR_INVALID_ARG;
    if (y == nullptr && (gate != nullptr || w_post != nullptr || scale != nullptr || dy != nullptr))
      return RAPT_ERR_INVALID_ARG;
    if ((dgate != nullptr && gate == nullptr) || (dw_pre != nullptr && dh == nullptr)) return RAPT_ERR_INVALID_ARG;
  }
  if (any_off16({dr, dh, x, y, gate, w_post, scale, w_pre, dx, dy, dgate, dw_post, dscale, dw_pre}))
    return RAPT_ERR_INVALID_ARG;
  if (any_same({dx, dy, dgate, dw_post, dscale, dw_pre}) ||
      aliases({dw_post, dscale, dw_pre}, {w_post, scale, w_pre}))
    return RAPT_ERR_INVALID_ARG;
  const bool sums = dw_post != nullptr || dscale != nullptr || dw_pre != nullptr;
  const size_t need = sums ? rapt::residual_norm_ws_bytes(T, D, to_dt(dtype)) : 0;
  if (workspace_bytes < need || (need > 0 && (workspace == nullptr || off16(workspace)))) return RAPT_ERR_WORKSPACE;
  rapt::ResidualNormArgs a{};
  a.x = dh != nullptr ? x : nullptr;
  a.y = y; a.gate = gate;
  a.w_post = w_post; a.scale = scale; a.w_pre = w_pre;
  a.dr = dr; a.dh = dh;
  a.dx = dx; a.dy = dy; a.dgate = dgate;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.T = T; a.D = D; a.act = to_act(act); a.eps = eps;
  return from_cuda(
      rapt::launch_residual_norm_bwd(to_dt(dtype), a, dw_post, dscale, dw_pre, as_stream(stream)));
}

rapt_status rapt_glu_fwd(const void* x, const void* w_gate, const void* w_up, int32_t M, int32_t F,
                         int32_t K, rapt_act act, void* h, uint32_t* dev_status, rapt_stream_t stream) {
  if (!known_act(act)) return RAPT_ERR_UNSUPPORTED;
  const rapt_status st = check_gemm(M, F, K);
  if (st != RAPT_OK) return st;
  if (w_gate == nullptr || w_up == nullptr || (M > 0 && (x == nullptr || h == nullptr))) return RAPT_ERR_INVALID_ARG;
  if (any_off16({x, w_gate, w_up, h}) || bad_status_word(dev_status)) return RAPT_ERR_INVALID_ARG;
  if (aliases({h}, {x, w_gate, w_up})) return RAPT_ERR_INVALID_ARG;
  if (M == 0) return RAPT_OK;
  rapt::GluArgs g{};
  g.x = x; g.w_gate = w_gate; g.w_up = w_up;
  g.M = M; g.F = F; g.K = K; g.act = to_act(act);
  g.dev_status = dev_status;
  return from_cuda(rapt::launch_glu_fwd(g, h, as_stream(stream)));
}

size_t rapt_glu_bwd_workspace_size(int32_t M, int32_t F, int32_t K) {
  if (check_gemm(M, F, K) != RAPT_OK || M == 0) return 0;
  return rapt::glu_bwd_ws_bytes(M, F, K, true, true);
}

rapt_status rapt_glu_bwd(const void* dh, const void* x, const void* w_gate, const void* w_up, int32_t M,
                         int32_t F, int32_t K, rapt_act act, void* dx, void* dw_gate, void* dw_up,
                         uint32_t* dev_status, void* workspace, size_t workspace_bytes,
                         rapt_stream_t stream) {
  if (!known_act(act)) return RAPT_ERR_UNSUPPORTED;
  rapt_status st = check_gemm(M, F, K);
  if (st != RAPT_OK) return st;
  if (w_gate == nullptr || w_up == nullptr || (M > 0 && (x == nullptr || dh == nullptr))) return RAPT_ERR_INVALID_ARG;
  if ((dx == nullptr && dw_gate == nullptr) || (dw_gate == nullptr) != (dw_up == nullptr)) return RAPT_ERR_INVALID_ARG;
  if (any_off16({dh, x, w_gate, w_up, dx, dw_gate, dw_up}) || bad_status_word(dev_status)) return RAPT_ERR_INVALID_ARG;
  if (any_same({dx, dw_gate, dw_up}) || aliases({dx, dw_gate, dw_up}, {dh, x, w_gate, w_up}))
    return RAPT_ERR_INVALID_ARG;
  if (M == 0) {
    const long long n = static_cast<long long>(F) * K;
    st = zero_bf16(dw_gate, n, stream);
    return st != RAPT_OK ? st : zero_bf16(dw_up, n, stream);
  }
  const size_t need = rapt::glu_bwd_ws_bytes(M, F, K, dx != nullptr, dw_gate != nullptr);
  if (workspace_bytes < need || workspace == nullptr || off16(workspace)) return RAPT_ERR_WORKSPACE;
  rapt::GluArgs g{};
  g.x = x; g.w_gate = w_gate; g.w_up = w_up;
  g.M = M; g.F = F; g.K = K; g.act = to_act(act);
  g.dev_status = dev_status;
  return from_cuda(rapt::launch_glu_bwd(g, dh, dx, dw_gate, dw_up, workspace, as_stream(stream)));
}

size_t rapt_linear_bwd_workspace_size(int32_t M, int32_t N, int32_t K) {
  if (check_gemm(M, N, K) != RAPT_OK || M == 0) return 0;
  return rapt::linear_bwd_ws_bytes(M, N, K, true, true);
}

rapt_status rapt_linear_bwd(const void* dy, const void* x, const void* w, int32_t M, int32_t N,
                            int32_t K, void* dx, void* dw, uint32_t* dev_status, void* workspace,
                            size_t workspace_bytes, rapt_stream_t stream) {
  const rapt_status st = check_gemm(M, N, K);
  if (st != RAPT_OK) return st;
  if (dx == nullptr && dw == nullptr) return RAPT_ERR_INVALID_ARG;
  if (M > 0 && (dy == nullptr || (dw != nullptr && x == nullptr))) return RAPT_ERR_INVALID_ARG;
  if (dx != nullptr && w == nullptr) return RAPT_ERR_INVALID_ARG;
  if (any_off16({dy, x, w, dx, dw}) || bad_status_word(dev_status)) return RAPT_ERR_INVALID_ARG;
  if (any_same({dx, dw}) || aliases({dx, dw}, {dy, x, w})) return RAPT_ERR_INVALID_ARG;
  if (M == 0) return zero_bf16(dw, static_cast<long long>(N) * K, stream);
  const size_t need = rapt::linear_bwd_ws_bytes(M, N, K, dx != nullptr, dw != nullptr);
  if (workspace_bytes < need || (need > 0 && (workspace == nullptr || off16(workspace)))) return RAPT_ERR_WORKSPACE;
  return from_cuda(
      rapt::launch_linear_bwd(dy, x, w, dx, dw, M, N, K, workspace, dev_status, as_stream(stream)));
}

}  // extern "C"
