// Forward of the residual norm; the mathematics and the layout of the work are in residual_norm.cuh.
#include "residual_norm.cuh"

namespace rapt {
namespace {

using namespace rn;

template <typename T, Rows R, int NC, int STAGES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) residual_norm_fwd_kernel(const ResidualNormArgs a, int tpr) {
  using C = Cols<T, R, NC, (STAGES > 0)>;
  __shared__ __align__(16) float red[2][32][8];
  extern __shared__ __align__(16) uint8_t ring[];
  int half = 0;
  const int tx = threadIdx.x % tpr, slots = blockDim.x / tpr, D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const C in(tx, tpr, D, static_cast<long>(blockIdx.x) * slots + threadIdx.x / tpr);
  Quad ws[NC], wpre[NC];
  load_gains(a, in, ws, wpre);
  const bool post = a.w_post != nullptr, gated = a.gate != nullptr, joined = a.y != nullptr;
  const long step = static_cast<long>(gridDim.x) * slots, step_off = step * D;
  long row = static_cast<long>(blockIdx.x) * slots + threadIdx.x / tpr, off = row * D;
  uint8_t* const mine = ring + threadIdx.x * C::kBytes;
  const uint32_t stage_bytes = blockDim.x * C::stride(kFwdTensors);
  const auto at = [&](const void* t, long o, bool live) { return t != nullptr && live ? static_cast<const T*>(t) + o : nullptr; };
  const auto fetch = [&](uint8_t* st, long rw, long o) {
    if (rw < a.T) {
      in.fetch(st, 0, static_cast<const T*>(a.x) + o);
      if (joined) in.fetch(st, 1, static_cast<const T*>(a.y) + o);
      if (gated) in.fetch(st, 2, static_cast<const T*>(a.gate) + o);
    } else {
#pragma unroll
      for (int k = 0; k < kFwdTensors; ++k) in.clear(st, k);
    }
    commit_copies();
  };
  // this thread's part of the sum of y^2 over a row
  const auto y_square = [&](uint8_t* st, const T* y_row) {
    Quad y[NC];
    in.read(st, 1, y_row, y);
    float2 q = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) q = dot4(y[c], y[c], q);
    return q.x + q.y;
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
#pragma unroll
    for (int k = 0; k < kFwdTensors; ++k) in.clear(mine + s * stage_bytes, k);
    fetch(mine + s * stage_bytes, row + s * step, off + s * step_off);
  }
  float sg = 1.f;
  if (post) {
    wait_copies<STAGES - 1>();
    float q[1] = {y_square(mine, at(a.y, off, row < a.T))};
    row_sum<1>(q, tpr, red, half);
    sg = inv_root(fmaf(q[0], inv_d, a.eps));
  }
  uint32_t s = 0;  // offset of the stage
  // the rows of a warp end together: those past T are zeros and not stored
  for (long first = static_cast<long>(blockIdx.x) * slots; first < a.T;
       first += step, row += step, off += step_off) {
    const bool live = row < a.T;
    const uint32_t next = s + stage_bytes == STAGES * stage_bytes ? 0 : s + stage_bytes;
    uint8_t* const st = mine + s;
    wait_copies<STAGES - 2>();  // this row and the next
    Quad r[NC], n[NC], z[NC];
    if (gated) in.read(st, 2, at(a.gate, off, live), z);
    act_cols<false>(gated, a.act, z, z, z);
    in.read(st, 0, at(a.x, off, live), r);
    in.read(st, 1, at(a.y, off, live), n);
    float2 sq = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      r[c] = fma4(n[c] * sg * z[c], ws[c], r[c]);
      sq = dot4(r[c], r[c], sq);
    }
    in.write(a.r != nullptr && live ? static_cast<T*>(a.r) + off : nullptr, r);
    fetch(st, row + STAGES * step, off + STAGES * step_off);
    float q[2] = {sq.x + sq.y, post ? y_square(mine + next, at(a.y, off + step_off, row + step < a.T)) : 0.f};
    row_sum<2>(q, tpr, red, half);
    if (post) sg = inv_root(fmaf(q[1], inv_d, a.eps));
    const float rho = inv_root(fmaf(q[0], inv_d, a.eps));
#pragma unroll
    for (int c = 0; c < NC; ++c) r[c] = r[c] * rho * wpre[c];
    in.write(a.h != nullptr && live ? static_cast<T*>(a.h) + off : nullptr, r);
    s = next;
  }
}

template <typename T, Rows R, int NC, int STAGES, int MAXT, int MINB>
cudaError_t go(const ResidualNormArgs& a, const RowShape& s, cudaStream_t stream) {
  const size_t smem = ring_bytes<T, R, NC>(s, STAGES, kFwdTensors);
  if constexpr (STAGES > 0 && NC > 2) {  // eight columns a thread always fit
    if (smem > kSmemMost) return go<T, R, NC, 0, MAXT, MINB>(a, s, stream);
  }
  int grid = 0;
  return launch_rows<residual_norm_fwd_kernel<T, R, NC, STAGES, MAXT, MINB>>(a, s, smem, 1 << 30, kMore<T, R> + 1,
                                                                             &grid, stream);
}
// Eight columns a thread up to D = 8192, then sixteen, or twenty-four of rows that take a few columns of
// another one with them (sixteen would need more than 1024 threads from D = 16378 on). Two stages of the ring for the narrow rows, three
// for the wide ones where they fit: bf16, % of the copy rate with 2 / 3 / 4 stages: D = 256: 92 / 81 /
// 79, D = 2048: 89 / 90 / 87, D = 4096: 88 / 92 / 90.
template <typename T, Rows R>
cudaError_t pick(const ResidualNormArgs& a, cudaStream_t stream) {
  constexpr int kS = sizeof(T) == 2 ? 3 : 2, kPlus = kMore<T, R>;
  const bool eight = a.D + kPlus <= 8192;
  constexpr int kWide = R == Rows::Whole ? 16 : 24;
  const RowShape s = row_shape(a.D, eight ? 8 : kWide, kPlus);
  if (!eight) return go<T, R, kWide / 4, 2, R == Rows::Whole ? 1024 : 704, 1>(a, s, stream);
  if (s.threads <= 256) return go<T, R, 2, 2, 256, 4>(a, s, stream);
  if (s.threads <= 512) return go<T, R, 2, kS, 512, 2>(a, s, stream);
  return go<T, R, 2, kS, 1024, 1>(a, s, stream);
}
template <typename T>
cudaError_t pick_rows(const ResidualNormArgs& a, cudaStream_t stream) {
  return whole_rows<T>(a.D) ? pick<T, Rows::Whole>(a, stream) : pick<T, Rows::Shifted>(a, stream);
}

}  // namespace

cudaError_t launch_residual_norm_fwd(DType dt, const ResidualNormArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return dt == DType::F32 ? pick_rows<float>(a, stream) : pick_rows<__nv_bfloat16>(a, stream);
}

}  // namespace rapt
