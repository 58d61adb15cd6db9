// Forward of the residual norm; the mathematics and the layout of the work are in residual_norm.cuh.
#include "residual_norm.cuh"

namespace rapt {
namespace {

using namespace rn;

template <typename T, Rows R, int NC, int STAGES, bool AHEAD, int MAXT, int MINB>
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
  // the ring: STAGES rows of x, gate and y; AHEAD: y apart, and a row further ahead than the others, so
  // that no row but the one in question has to have arrived
  constexpr int kYSlot = AHEAD ? 0 : 2;
  uint8_t* const mine = ring + threadIdx.x * C::kBytes;
  const uint32_t stage_bytes = blockDim.x * C::stride(AHEAD ? 2 : 3), y_bytes = blockDim.x * C::stride(1);
  uint8_t* const mine_y = mine + (AHEAD ? STAGES * stage_bytes : 0);
  const auto at = [&](const void* t, long o, bool live) { return t != nullptr && live ? static_cast<const T*>(t) + o : nullptr; };
  const auto fetch_y = [&](uint8_t* st, long rw, long o) {
    if (rw >= a.T)
      in.clear(st, 0);
    else if (joined)
      in.fetch(st, 0, static_cast<const T*>(a.y) + o);
  };
  const auto fetch = [&](uint8_t* st, uint8_t* st_y, long rw, long o) {
    if (rw < a.T) {
      in.fetch(st, 0, static_cast<const T*>(a.x) + o);
      if (!AHEAD && joined) in.fetch(st, 2, static_cast<const T*>(a.y) + o);
      if (gated) in.fetch(st, 1, static_cast<const T*>(a.gate) + o);
    } else {
#pragma unroll
      for (int k = 0; k < (AHEAD ? 2 : 3); ++k) in.clear(st, k);
    }
    if (AHEAD) fetch_y(st_y, rw + step, o + step_off);
    commit_copies();
  };
  // this thread's part of the sum of y^2 over a row
  const auto y_square = [&](uint8_t* st, const T* y_row) {
    Quad y[NC];
    in.read(st, kYSlot, y_row, y);
    float2 q = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) q = dot4(y[c], y[c], q);
    return q.x + q.y;
  };
  if constexpr (AHEAD) {
    in.clear(mine_y, 0);
    fetch_y(mine_y, row, off);
  }
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
#pragma unroll
    for (int k = 0; k < (AHEAD ? 2 : 3); ++k) in.clear(mine + s * stage_bytes, k);
    if (AHEAD) in.clear(mine_y + (s + 1) * y_bytes, 0);
    fetch(mine + s * stage_bytes, mine_y + (s + 1) * y_bytes, row + s * step, off + s * step_off);
  }
  float sg = 1.f;
  if (post) {
    wait_copies<STAGES - 1>();
    float q[1] = {y_square(mine_y, at(a.y, off, row < a.T))};
    row_sum<1>(q, tpr, red, half);
    sg = inv_root(fmaf(q[0], inv_d, a.eps));
  }
  uint32_t s = 0, sy = 0;  // offsets of the stage and, AHEAD, of the row's y
  // the rows of a warp end together: those past T are zeros and not stored
  for (long first = static_cast<long>(blockIdx.x) * slots; first < a.T;
       first += step, row += step, off += step_off) {
    const bool live = row < a.T;
    const uint32_t next = s + stage_bytes == STAGES * stage_bytes ? 0 : s + stage_bytes;
    const uint32_t next_y = sy == STAGES * y_bytes ? 0 : sy + y_bytes;
    uint8_t *const st = mine + s, *const st_y = AHEAD ? mine_y + sy : st;
    wait_copies<STAGES - 2 + AHEAD>();  // this row and the next one's y
    Quad r[NC], n[NC], z[NC];
    if (gated) in.read(st, 1, at(a.gate, off, live), z);
    act_cols<false>(gated, a.act, z, z, z);
    in.read(st, 0, at(a.x, off, live), r);
    in.read(st_y, kYSlot, at(a.y, off, live), n);
    float2 sq = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      r[c] = fma4(n[c] * sg * z[c], ws[c], r[c]);
      sq = dot4(r[c], r[c], sq);
    }
    in.write(a.r != nullptr && live ? static_cast<T*>(a.r) + off : nullptr, r);
    if (STAGES > 0) fetch(st, st_y, row + STAGES * step, off + STAGES * step_off);
    float q[2] = {sq.x + sq.y, post ? y_square(AHEAD ? mine_y + next_y : mine + next, at(a.y, off + step_off, row + step < a.T)) : 0.f};
    row_sum<2>(q, tpr, red, half);
    if (post) sg = inv_root(fmaf(q[1], inv_d, a.eps));
    const float rho = inv_root(fmaf(q[0], inv_d, a.eps));
#pragma unroll
    for (int c = 0; c < NC; ++c) r[c] = r[c] * rho * wpre[c];
    in.write(a.h != nullptr && live ? static_cast<T*>(a.h) + off : nullptr, r);
    s = next;
    sy = next_y;
  }
}

template <typename T, Rows R, int NC, int STAGES, bool AHEAD, int MAXT, int MINB>
cudaError_t go(const ResidualNormArgs& a, const RowShape& s, cudaStream_t stream) {
  const size_t smem = ring_bytes<T, R, NC>(s, STAGES, kFwdTensors) + (AHEAD ? ring_bytes<T, R, NC>(s, 1, 1) : 0);
  int grid = 0;
  return launch_rows<residual_norm_fwd_kernel<T, R, NC, STAGES, AHEAD, MAXT, MINB>>(a, s, smem, 1 << 30,
                                                                                    kMore<T, R> + 1, &grid, stream);
}
// Columns a thread, and the ring. us of 128 MiB a tensor (columns a thread / stages, + where y is ahead):
//   bf16  D = 2048: 8/2 113, 16/2+ 119;  3584: 16/2+ 111, 8/3 118;  5120: 16/2+ 110, 8/3 126;
//         10240: 24/2+ 122, 16/2+ 172;  12288: 24/2+ 107, 16/3 137;  16384: 16/2+ 132, 24/1+ 146
//         D = 1001, 4098 (rows that are no whole vectors): 16/2+ 132, 160, 8/3 152, 197
//   fp32  D = 512: 16/1+ 109, 8/2 114;  1024: 8/2 113, 16/1+ 111;  5120: 8/2 105, 16/1+ 114;
//         6144: 16/1+ 105, 8/2 112;  12288: 24/1+ 119, 16 without a ring 145
//         D = 257, 1001, 4098: 16/1+ 127, 115, 111, 8/2 183, 122, 133
template <typename T, Rows R>
cudaError_t pick(const ResidualNormArgs& a, cudaStream_t stream) {
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kMoreCols = kMore<T, R>, kS = kF32 ? 1 : 2;
  const int n = a.D + kMoreCols, eight = kF32 ? (kMoreCols > 0 ? 4096 : 5120) : kMoreCols > 0 ? 0 : 2048;
  const int ept = n <= 256 || (n > 512 && n <= eight) ? 8 : n <= 8192 ? 16 : n <= 12288 || kMoreCols > 0 ? 24 : 16;
  const RowShape s = row_shape(a.D, ept, kMoreCols);
  if (ept == 8) {
    if (s.threads <= 256) return go<T, R, 2, 2, false, 256, 4>(a, s, stream);
    if constexpr (kF32) {
      if (s.threads <= 512) return go<T, R, 2, 2, false, 512, 2>(a, s, stream);
      if constexpr (R == Rows::Whole) return go<T, R, 2, 2, false, 640, 1>(a, s, stream);
    }
  }
  if (ept == 24) {
    if (s.threads <= 512) return go<T, R, 6, kS, true, 512, 1>(a, s, stream);
    if constexpr (R == Rows::Shifted) return go<T, R, 6, kS - 1, !kF32, 704, 1>(a, s, stream);
  }
  if (s.threads <= 128) return go<T, R, 4, 1, true, 128, 4>(a, s, stream);
  if constexpr (!kF32)
    if (s.threads <= 256) return go<T, R, 4, kS, true, 256, 2>(a, s, stream);
  if (s.threads <= 320) return go<T, R, 4, kS, true, 320, 2>(a, s, stream);
  if (s.threads <= 512) return go<T, R, 4, kS, true, 512, 1>(a, s, stream);
  if constexpr (R == Rows::Whole) return go<T, R, 4, kF32 ? 0 : kS, !kF32, 1024, 1>(a, s, stream);
  return cudaErrorInvalidConfiguration;  // not reached
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
