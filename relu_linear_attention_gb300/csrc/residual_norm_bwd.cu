// Backward of the residual norm; the mathematics and the layout of the work are in residual_norm.cuh.
#include "residual_norm.cuh"
#include "tc_utils.cuh"

namespace rapt {
namespace {

using namespace rn;

// Partial column sums of CTA b at part[(b * 2 + k) * D + column], k = 0: G, 1: dw_pre.
template <typename T, Rows R, int NC, int STAGES, bool AHEAD, int GAINS, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) residual_norm_bwd_kernel(const ResidualNormArgs a, int tpr) {
  using C = Cols<T, R, NC, (STAGES > 0)>;
  __shared__ __align__(16) float red[2][32][8];
  extern __shared__ __align__(16) uint8_t ring[];
  int half = 0;
  const int tx = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const C in(tx, tpr, D, static_cast<long>(blockIdx.x) * slots + threadIdx.x / tpr);
  // w_post s and w_pre of this thread's columns: the first GAINS of them in shared memory behind the ring
  // where they would spill (bf16, D = 8192: 315 us with both in registers, 258 with none)
  Quad ws_kept[GAINS > 0 ? 1 : NC], wpre_kept[GAINS > 1 ? 1 : NC];
  uint8_t* const gains = ring + blockDim.x * (STAGES * C::stride(kBwdTensors) + AHEAD * C::stride(1)) + threadIdx.x * 16;
  {
    Quad ws[NC], wpre[NC];
    load_gains(a, in, ws, wpre);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (GAINS > 0)
        *reinterpret_cast<Quad*>(gains + c * 16 * blockDim.x) = ws[c];
      else
        ws_kept[c] = ws[c];
      if constexpr (GAINS > 1)
        *reinterpret_cast<Quad*>(gains + (NC + c) * 16 * blockDim.x) = wpre[c];
      else
        wpre_kept[c] = wpre[c];
    }
  }
  const auto ws = [&](int c) {
    if constexpr (GAINS > 0)
      return *reinterpret_cast<const Quad*>(gains + c * 16 * blockDim.x);
    else
      return ws_kept[c];
  };
  const auto wpre = [&](int c) {
    if constexpr (GAINS > 1)
      return *reinterpret_cast<const Quad*>(gains + (NC + c) * 16 * blockDim.x);
    else
      return wpre_kept[c];
  };
  const bool post = a.w_post != nullptr, gated = a.gate != nullptr, joined = a.y != nullptr, normed = a.dh != nullptr;
  Quad gg[NC], gpre[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) gg[c] = gpre[c] = quad(0.f);
  const long step = static_cast<long>(gridDim.x) * slots, step_off = step * D;
  long row = static_cast<long>(blockIdx.x) * slots + slot, off = row * D;
  // the ring: STAGES rows of dh, x, gate, dr and y; AHEAD: y apart, and a row further ahead than the
  // others, so that no row but the one in question has to have arrived
  constexpr bool kEarly = STAGES == 1;  // x and gate of the next row are fetched when this one's are read
  constexpr int kYSlot = AHEAD ? 0 : 4;
  uint8_t* const mine = ring + threadIdx.x * C::kBytes;
  const uint32_t stage_bytes = blockDim.x * C::stride(AHEAD ? 4 : 5), y_bytes = blockDim.x * C::stride(1);
  uint8_t* const mine_y = mine + (AHEAD ? STAGES * stage_bytes : 0);
  const auto at = [&](const void* t, long o, bool live) { return t != nullptr && live ? static_cast<const T*>(t) + o : nullptr; };
  // tensor slots of a stage: dh, dr, x, gate (, y); x and gate are read before the reduction only
  const auto fetch_early = [&](uint8_t* st, long rw, long o) {
    if (rw < a.T) {
      if (normed) in.fetch(st, 2, static_cast<const T*>(a.x) + o);
      if (gated) in.fetch(st, 3, static_cast<const T*>(a.gate) + o);
    } else {
      in.clear(st, 2);
      in.clear(st, 3);
    }
  };
  const auto fetch_y = [&](uint8_t* st, long rw, long o) {
    if (rw >= a.T)
      in.clear(st, 0);
    else if (joined)
      in.fetch(st, 0, static_cast<const T*>(a.y) + o);
  };
  const auto fetch = [&](uint8_t* st, uint8_t* st_y, long rw, long o) {
    if (rw < a.T) {
      if (normed) {
        in.fetch(st, 0, static_cast<const T*>(a.dh) + o);
        if (!kEarly) in.fetch(st, 2, static_cast<const T*>(a.x) + o);
      }
      if (!AHEAD && joined) in.fetch(st, 4, static_cast<const T*>(a.y) + o);
      if (!kEarly && gated) in.fetch(st, 3, static_cast<const T*>(a.gate) + o);
      if (a.dr != nullptr) in.fetch(st, 1, static_cast<const T*>(a.dr) + o);
    } else {
#pragma unroll
      for (int k = 0; k < (AHEAD ? 4 : 5); ++k)
        if (!kEarly || k < 2) in.clear(st, k);
    }
    if (AHEAD) fetch_y(st_y, rw + step, o + step_off);
    commit_copies();
  };
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
    const long rw = row + s * step, o = off + s * step_off;
#pragma unroll
    for (int k = 0; k < (AHEAD ? 4 : 5); ++k) in.clear(mine + s * stage_bytes, k);
    if (AHEAD) in.clear(mine_y + (s + 1) * y_bytes, 0);
    if (kEarly) fetch_early(mine + s * stage_bytes, rw, o);
    fetch(mine + s * stage_bytes, mine_y + (s + 1) * y_bytes, rw, o);
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
    Quad r[NC], av[NC], da[NC];  // x + e, act(z), act'(z): kept over the reduction
    float q[6];
    {
      Quad e[NC], t[NC], d[NC];
      if (gated) in.read(st, 3, at(a.gate, off, live), t);
      act_cols<true>(gated, a.act, t, av, da);
      in.read(st_y, kYSlot, at(a.y, off, live), e);
      in.read(st, 2, at(normed ? a.x : nullptr, off, live), r);
      if (kEarly) fetch_early(st, row + step, off + step_off);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        e[c] = e[c] * sg * ws(c) * av[c];
        r[c] = fma4(e[c], quad(1.f), r[c]);
      }
      in.read(st, 0, at(a.dh, off, live), t);
      in.read(st, 1, at(a.dr, off, live), d);
      float2 rr = both(0.f), tr = rr, ed = rr, et = rr, er = rr;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        t[c] = t[c] * wpre(c);
        rr = dot4(r[c], r[c], rr);
        tr = dot4(t[c], r[c], tr);
        ed = dot4(e[c], d[c], ed);
        et = dot4(e[c], t[c], et);
        er = dot4(e[c], r[c], er);
      }
      q[0] = rr.x + rr.y;
      q[1] = tr.x + tr.y;
      q[2] = ed.x + ed.y;
      q[3] = et.x + et.y;
      q[4] = er.x + er.y;
    }
    q[5] = post ? y_square(AHEAD ? mine_y + next_y : mine + next, at(a.y, off + step_off, row + step < a.T)) : 0.f;
    row_sum<6>(q, tpr, red, half);
    const float rho = normed ? inv_root(fmaf(q[0], inv_d, a.eps)) : 0.f;
    // mean(t rh), mean(u yh). rho = 0 (no dh, or sum r^2 overflowed): rh = 0, and the sums with r, which may have
    // overflowed, too, do not count. (To form them again where one overflows for rho > 0 made every call 4 to
    // 16 % slower as another turn of this code, 16 to 38 % in bf16 as a path of its own: registers.)
    const float m = rho > 0.f ? rho * q[1] * inv_d : 0.f;
    const float my = post ? inv_d * (rho > 0.f ? q[2] + rho * (q[3] - rho * m * q[4]) : q[2]) : 0.f;
    Quad g[NC], y[NC], t[NC];
    in.read(st, 1, at(a.dr, off, live), g);
    in.read(st, 0, at(a.dh, off, live), t);
    in.read(st_y, kYSlot, at(a.y, off, live), y);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const Quad rh = r[c] * rho;
      gpre[c] = fma4(t[c], rh, gpre[c]);
      g[c] = fma4(quad(rho), fma4(rh, quad(-m), t[c] * wpre(c)), g[c]);
    }
    in.write(a.dx != nullptr && live ? static_cast<T*>(a.dx) + off : nullptr, g);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      y[c] = y[c] * sg;  // yh
      const Quad ag = av[c] * g[c];
      gg[c] = fma4(ag, y[c], gg[c]);
      const Quad w = ws(c);
      da[c] = da[c] * g[c] * (y[c] * w);
      g[c] = fma4(y[c], quad(-my), w * ag) * sg;
    }
    in.write(a.dgate != nullptr && live ? static_cast<T*>(a.dgate) + off : nullptr, da);
    in.write(a.dy != nullptr && live ? static_cast<T*>(a.dy) + off : nullptr, g);
    if (STAGES > 0) fetch(st, st_y, row + STAGES * step, off + STAGES * step_off);
    if (post) sg = inv_root(fmaf(q[5], inv_d, a.eps));
    s = next;
    sy = next_y;
  }
  if (a.part == nullptr) return;
  tc::grid_launch_dependents();  // the sum over the CTAs may be made ready
  float* out = a.part + static_cast<long>(blockIdx.x) * 2 * D;
  if (slots == 1) {
    in.put_sums(out, gg);
    in.put_sums(out + D, gpre);
    return;
  }
  // the slots' sums meet in shared memory, where no copy is on its way any more
  wait_copies<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
  in.put_sums(sums + slot * 2 * D, gg);
  in.put_sums(sums + slot * 2 * D + D, gpre);
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += blockDim.x) {
    float v = 0.f;
    for (int i = 0; i < slots; ++i) v += sums[i * 2 * D + e];
    out[e] = v;
  }
}

// The gain gradients: the CTAs' partial sums added in a fixed order. blockIdx.y picks G (dw_post = s G,
// dscale = w_post G) or dw_pre; 32 x 32 threads take 32 columns: thread (c, q) adds partials q, q + 32,
// ..., then the 32 sums of a column are added in order of q. No partials (T = 0) gives zeros.
struct GainGrads {
  const float *part, *w_post, *scale;
  float *dw_post, *dscale, *dw_pre;
  int nparts, D;
};
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(const GainGrads a) {
  __shared__ float s[32][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  tc::grid_dep_wait();  // the partials of the launch before this one
  if (c < a.D) {
#pragma unroll 8
    for (int b = threadIdx.y; b < a.nparts; b += 32) v += a.part[(static_cast<long>(b) * 2 + k) * a.D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= a.D) return;
  float t = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) t += s[q][threadIdx.x];
  if (k == 1) {
    if (a.dw_pre != nullptr) a.dw_pre[c] = t;
    return;
  }
  if (a.dw_post != nullptr) a.dw_post[c] = a.scale != nullptr ? a.scale[c] * t : t;
  if (a.dscale != nullptr) a.dscale[c] = a.w_post != nullptr ? a.w_post[c] * t : t;
}

template <typename T, Rows R, int NC, int STAGES, bool AHEAD, int GAINS, int MAXT, int MINB>
cudaError_t go(const ResidualNormArgs& a, const RowShape& s, int* grid, cudaStream_t stream) {
  size_t smem = ring_bytes<T, R, NC>(s, STAGES, kBwdTensors) + (AHEAD ? ring_bytes<T, R, NC>(s, 1, 1) : 0) +
                static_cast<size_t>(s.threads) * GAINS * NC * sizeof(Quad);
  // the slots' column sums meet where the ring was
  if (s.tpr <= 32) smem = std::max(smem, static_cast<size_t>(s.threads / s.tpr) * 2 * a.D * 4);
  return launch_rows<residual_norm_bwd_kernel<T, R, NC, STAGES, AHEAD, GAINS, MAXT, MINB>>(
      a, s, smem, max_parts(s), kMore<T, R> + 1, grid, stream);
}
// Columns a thread, the ring and the gains in shared memory. us of 128 MiB a tensor, columns a thread /
// stages, + where y is ahead, g1 or g2 with gains in shared memory, the best choices and others:
//   bf16  D = 2560: 8/4 two CTAs an SM 197, one 269;  5120: 16/3 229, 16/2 314;  6144: 16/3 210, 16/2 282;
//         8192: 16/2 g2 258, 16/2 315, 32/1+ 326;  12288: 24/1+ g1 358, 24/1+ 422, 16 without a ring 683;
//         16384: 32 without a ring, g2 635, 32/1+ 690
//   fp32  D = 2560: 8/2+ two CTAs an SM 173, 8/2 one 256;  4096: 8/2+ 190, 8/2 202;  5120: 16/2+ 204,
//         16/2 247;  7168: 16/1+ g2 194, 16/1+ 271;  8192: 16/1+ g1 233, 16/1+ 258, without a ring 299;
//         12288: 24 without a ring, g2 387, 24 411, 16 544;  16384: 32, g2 504, 32 562
template <typename T, Rows R>
cudaError_t pick(const ResidualNormArgs& a, int* grid, cudaStream_t stream) {
  constexpr bool kF32 = sizeof(T) == 4;
  const RowShape s = bwd_shape(a.D, kMore<T, R>, kF32);
  if (s.ept == 8) {
    if (s.threads <= 256) return go<T, R, 2, kF32 ? 2 : 3, false, 0, 256, 2>(a, s, grid, stream);
    if (s.threads <= 320) return go<T, R, 2, kF32 ? 2 : 4, kF32, 0, 320, 2>(a, s, grid, stream);
    return go<T, R, 2, kF32 ? 2 : 4, kF32, 0, 512, 1>(a, s, grid, stream);
  }
  if constexpr (kF32) {
    if (s.ept == 16 && s.threads <= 320) return go<T, R, 4, 2, true, 0, 384, 1>(a, s, grid, stream);
    if (s.ept == 16 && s.threads <= 448) return go<T, R, 4, 1, true, 2, 448, 1>(a, s, grid, stream);
    if (s.ept == 16) return go<T, R, 4, 1, true, 1, 512, 1>(a, s, grid, stream);
    if (s.ept == 24 && s.threads <= 512) return go<T, R, 6, 0, false, 2, 512, 1>(a, s, grid, stream);
  } else {
    if (s.ept == 16 && s.threads <= 128) return go<T, R, 4, 3, false, 0, 128, 3>(a, s, grid, stream);
    if (s.ept == 16 && s.threads <= 384) return go<T, R, 4, 3, false, 0, 384, 1>(a, s, grid, stream);
    if (s.ept == 16) return go<T, R, 4, 2, false, 2, 512, 1>(a, s, grid, stream);
    if (s.ept == 24 && s.threads <= 448) return go<T, R, 6, 1, true, 2, 448, 1>(a, s, grid, stream);
    if (s.ept == 24 && s.threads <= 512) return go<T, R, 6, 1, true, 1, 512, 1>(a, s, grid, stream);
  }
  if constexpr (R == Rows::Whole)
    return go<T, R, 8, 0, false, 2, 512, 1>(a, s, grid, stream);
  else
    return go<T, R, 6, 0, false, 2, 704, 1>(a, s, grid, stream);
}
template <typename T>
cudaError_t pick_rows(const ResidualNormArgs& a, int* grid, cudaStream_t stream) {
  return whole_rows<T>(a.D) ? pick<T, Rows::Whole>(a, grid, stream) : pick<T, Rows::Shifted>(a, grid, stream);
}

}  // namespace

size_t residual_norm_ws_bytes(long T, int D, DType dt) {
  const int vec = dt == DType::F32 ? kVec<float> : kVec<__nv_bfloat16>;
  const RowShape s = bwd_shape(D, D % vec == 0 ? 0 : vec - 1, dt == DType::F32);
  const long slots = s.threads / s.tpr;
  return static_cast<size_t>(std::min<long>((T + slots - 1) / slots, max_parts(s))) * 2 * D * 4;
}

cudaError_t launch_residual_norm_bwd(DType dt, const ResidualNormArgs& a, float* dw_post, float* dscale,
                                     float* dw_pre, cudaStream_t stream) {
  int grid = 0;
  if (a.T > 0) {
    const cudaError_t e =
        dt == DType::F32 ? pick_rows<float>(a, &grid, stream) : pick_rows<__nv_bfloat16>(a, &grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (dw_post == nullptr && dscale == nullptr && dw_pre == nullptr) return cudaSuccess;
  const GainGrads g{a.part, a.w_post, a.scale, dw_post, dscale, dw_pre, grid, a.D};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.D + 31) / 32, 2);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.T > 0 ? 1 : 0;  // not before what another call launched
  const cudaError_t e = cudaLaunchKernelEx(&cfg, residual_norm_sum_kernel, g);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rapt
