// Layer norm of rows of D values, and its gradients (sm_103a):
//   y = w xh + b,  xh = (x - m) r,  m = mean x,  r = (mean (x - m)^2 + eps)^(-1/2)
//   dx = r (g - mean g - xh mean(g xh)),  g = w dy,  dw = sum_rows dy xh,  db = sum_rows dy.
//
// HBM bound: the forward moves 2 tensors, the backward 3, each once. Rows lie and arrive as in the residual norm
// (residual_norm.cuh): a CTA takes a row at a time (8 to 32 lanes take a narrow one), the rows ahead are in
// flight in a ring in shared memory, each thread copies and reads its own columns alone. A row has one reduction:
// beside its own sums it carries sum x of the NEXT row, whose mean is then known when its turn comes, so that the
// variance is a sum of squared differences. With xc = x - m and the mean's own rounding error c = mean xc,
//   var = mean xc^2 - c^2,  xh = (xc - c) r,  sum g xh = r (sum g xc - c sum g):
// a row whose mean is 1e4 times its deviation keeps the bits that its values have. The backward's column sums
// stay in registers over the CTA's rows (fp32); a second small launch adds the CTAs' in a fixed order.
#include "residual_norm.cuh"
#include "tc_utils.cuh"

namespace rapt {
namespace {

using namespace rn;

__device__ __forceinline__ float sum4(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float2 add4(Quad a, float2 s) {
  return __fadd2_rn(a.p[1], __fadd2_rn(a.p[0], s));
}
__device__ __forceinline__ Quad minus(Quad a, float m) { return fma4(quad(1.f), a, quad(-m)); }

// Zeros where there is no column.
template <typename C, int NC>
__device__ __forceinline__ void clip(const C& in, Quad (&f)[NC]) {
  constexpr int Q = C::kPer / 4;  // quads of a piece
#pragma unroll
  for (int i = 0; i < C::kPieces; ++i) {
    const int e = in.col(i);
    if (e >= 0 && e + C::kPer <= in.D) continue;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float2& p = f[i * Q + q].p[k];
        p.x = in.has(e + 4 * q + 2 * k) ? p.x : 0.f;
        p.y = in.has(e + 4 * q + 2 * k + 1) ? p.y : 0.f;
      }
  }
}

template <bool BWD, typename T, Rows R, int NC, int STAGES, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) layer_norm_kernel(const LayerNormArgs a, int tpr) {
  using C = Cols<T, R, NC, true>;
  __shared__ __align__(16) float red[2][32][8];
  extern __shared__ __align__(16) uint8_t ring[];
  int half = 0;
  const int tx = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const long step = static_cast<long>(gridDim.x) * slots, step_off = step * D;
  long row = static_cast<long>(blockIdx.x) * slots + slot, off = row * D;
  const C in(tx, tpr, D, row);
  // the ring: x of STAGES + 1 rows, then dy of STAGES, each copied with the next row's x
  uint8_t* const mine = ring + threadIdx.x * C::kBytes;
  const uint32_t row_bytes = blockDim.x * C::stride(1);
  uint8_t* const mine_dy = mine + (STAGES + 1) * row_bytes;
  const auto fetch_x = [&](uint8_t* st, long rw, long o) {
    if (rw < a.T) in.fetch(st, 0, static_cast<const T*>(a.x) + o);
    else in.clear(st, 0);
  };
  const auto fetch = [&](uint8_t* st, uint8_t* st_dy, long rw, long o) {  // dy of row rw, x of the next
    if constexpr (BWD) {
      if (rw < a.T) in.fetch(st_dy, 0, static_cast<const T*>(a.dy) + o);
      else in.clear(st_dy, 0);
    }
    fetch_x(st, rw + step, o + step_off);
    commit_copies();
  };
  const auto read = [&](uint8_t* st, Quad (&f)[NC]) { in.read(st, 0, static_cast<const T*>(nullptr), f); };
  const auto x_sum = [&](uint8_t* st) {
    Quad x[NC];
    read(st, x);
    float2 q = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) q = add4(x[c], q);
    return sum4(q);
  };
  in.clear(mine, 0);
  fetch_x(mine, row, off);
  commit_copies();
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    in.clear(mine + (s + 1) * row_bytes, 0);
    if (BWD) in.clear(mine_dy + s * row_bytes, 0);
    fetch(mine + (s + 1) * row_bytes, mine_dy + s * row_bytes, row + s * step, off + s * step_off);
  }
  Quad w[NC], b[BWD ? 1 : NC], sw[BWD ? NC : 1], sb[BWD ? NC : 1];
  in.gain(a.w, w);
  if constexpr (BWD) {
#pragma unroll
    for (int c = 0; c < NC; ++c) sw[c] = sb[c] = quad(0.f);
  } else {
    in.gain(a.b, b);
    if (a.b == nullptr) {
#pragma unroll
      for (int c = 0; c < NC; ++c) b[c] = quad(0.f);
    }
  }
  float m;
  {
    wait_copies<STAGES>();
    float q[1] = {x_sum(mine)};
    row_sum<1>(q, tpr, red, half);
    m = q[0] * inv_d;
  }
  uint32_t s = 0, sd = 0;  // offsets of the row's x and dy
  // the rows of a warp end together: those past T are zeros and not stored
  for (long first = static_cast<long>(blockIdx.x) * slots; first < a.T;
       first += step, row += step, off += step_off) {
    const bool live = row < a.T;
    const uint32_t next = s == STAGES * row_bytes ? 0 : s + row_bytes;
    uint8_t *const st = mine + s, *const st_dy = mine_dy + sd;
    wait_copies<STAGES - 1>();  // this row and the next one's x
    Quad xc[NC];
    read(st, xc);
    float q[5];
    float2 s1 = both(0.f), s2 = s1, g1 = s1, g2 = s1;
#pragma unroll
    for (int c = 0; c < NC; ++c) xc[c] = minus(xc[c], m);
    clip(in, xc);
    if constexpr (BWD) {
      Quad g[NC];
      read(st_dy, g);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        g[c] = g[c] * w[c];
        g1 = add4(g[c], g1);
        g2 = dot4(g[c], xc[c], g2);
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      s1 = add4(xc[c], s1);
      s2 = dot4(xc[c], xc[c], s2);
    }
    q[0] = sum4(s1);
    q[1] = sum4(s2);
    q[2] = x_sum(mine + next);
    if constexpr (BWD) {
      q[3] = sum4(g1);
      q[4] = sum4(g2);
      row_sum<5>(q, tpr, red, half);
    } else {
      float p[3] = {q[0], q[1], q[2]};
      row_sum<3>(p, tpr, red, half);
      q[0] = p[0], q[1] = p[1], q[2] = p[2];
    }
    const float c0 = q[0] * inv_d;
    const float r = inv_root(fmaxf(fmaf(q[1], inv_d, -c0 * c0), 0.f) + a.eps);
    if constexpr (BWD) {
      const float mg = q[3] * inv_d, mgx = r * (q[4] - c0 * q[3]) * inv_d;
      Quad g[NC];
      read(st_dy, g);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const Quad xh = minus(xc[c], c0) * r;
        sw[c] = fma4(g[c], xh, sw[c]);
        sb[c] = fma4(g[c], quad(1.f), sb[c]);
        xc[c] = fma4(xh, quad(-mgx), minus(g[c] * w[c], mg)) * r;
      }
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c) xc[c] = fma4(minus(xc[c], c0) * r, w[c], b[c]);
    }
    in.write(a.out != nullptr && live ? static_cast<T*>(a.out) + off : nullptr, xc);
    fetch(st, st_dy, row + STAGES * step, off + STAGES * step_off);
    m = q[2] * inv_d;
    s = next;
    sd = sd + row_bytes == STAGES * row_bytes ? 0 : sd + row_bytes;
  }
  if constexpr (BWD) {
    if (a.part == nullptr) return;
    tc::grid_launch_dependents();  // the sum over the CTAs may be made ready
    float* out = a.part + static_cast<long>(blockIdx.x) * 2 * D;
    if (slots == 1) {
      in.put_sums(out, sw);
      in.put_sums(out + D, sb);
      return;
    }
    // the slots' sums meet in shared memory, where no copy is on its way any more
    wait_copies<0>();
    __syncthreads();
    float* sums = reinterpret_cast<float*>(ring);
    in.put_sums(sums + slot * 2 * D, sw);
    in.put_sums(sums + slot * 2 * D + D, sb);
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < slots; ++i) v += sums[i * 2 * D + e];
      out[e] = v;
    }
  }
}

// The column sums: the CTAs' partials added in a fixed order. blockIdx.y picks dw or db; 32 x 32 threads take 32
// columns: thread (c, q) adds partials q, q + 32, ..., then the 32 sums of a column are added in order of q. No
// partials (T = 0) gives zeros.
__global__ void __launch_bounds__(1024)
    layer_norm_sum_kernel(const float* part, float* dw, float* db, int nparts, int D) {
  __shared__ float s[32][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* const out = k == 0 ? dw : db;
  float v = 0.f;
  tc::grid_dep_wait();  // the partials of the launch before this one
  if (c < D && out != nullptr) {
#pragma unroll 8
    for (int b = threadIdx.y; b < nparts; b += 32) v += part[(static_cast<long>(b) * 2 + k) * D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D || out == nullptr) return;
  float t = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) t += s[q][threadIdx.x];
  out[c] = t;
}

template <bool BWD, typename T, Rows R, int NC, int STAGES, int MAXT, int MINB>
cudaError_t go(const LayerNormArgs& a, const RowShape& s, int* grid, cudaStream_t stream) {
  size_t smem = ring_bytes<T, R, NC>(s, BWD ? 2 * STAGES + 1 : STAGES + 1, 1);
  // the slots' column sums meet where the ring was
  if (BWD && s.tpr <= 32) smem = std::max(smem, static_cast<size_t>(s.threads / s.tpr) * 2 * a.D * 4);
  return launch_rows<layer_norm_kernel<BWD, T, R, NC, STAGES, MAXT, MINB>>(a, s, smem, BWD ? max_parts(s) : 1 << 30,
                                                                           kMore<T, R> + 1, grid, stream);
}
// Columns a thread: 8 up to 4096, 16 up to 8192, 24 beyond.
inline RowShape shape(int D, int more) {
  const int n = D + more;
  return row_shape(D, n <= 4096 ? 8 : n <= 8192 ? 16 : 24, more);
}
template <bool BWD, typename T, Rows R>
cudaError_t pick(const LayerNormArgs& a, int* grid, cudaStream_t stream) {
  const RowShape s = shape(a.D, kMore<T, R>);
  constexpr bool kF32 = sizeof(T) == 4;
  if (s.ept == 8) {
    if (s.threads <= 256) return go<BWD, T, R, 2, kF32 ? 2 : 3, 256, BWD ? 3 : 4>(a, s, grid, stream);
    return go<BWD, T, R, 2, kF32 ? 2 : 3, 544, 1>(a, s, grid, stream);
  }
  if (s.ept == 16) return go<BWD, T, R, 4, 2, 544, 1>(a, s, grid, stream);
  return go<BWD, T, R, 6, BWD && kF32 ? 1 : 2, 704, 1>(a, s, grid, stream);
}
template <bool BWD, typename T>
cudaError_t pick_rows(const LayerNormArgs& a, int* grid, cudaStream_t stream) {
  return whole_rows<T>(a.D) ? pick<BWD, T, Rows::Whole>(a, grid, stream) : pick<BWD, T, Rows::Shifted>(a, grid, stream);
}

}  // namespace

size_t layer_norm_ws_bytes(long T, int D, DType dt) {
  const int vec = dt == DType::F32 ? kVec<float> : kVec<__nv_bfloat16>;
  const RowShape s = shape(D, D % vec == 0 ? 0 : vec - 1);
  const long slots = s.threads / s.tpr;
  return static_cast<size_t>(std::min<long>((T + slots - 1) / slots, max_parts(s))) * 2 * D * 4;
}

cudaError_t launch_layer_norm_fwd(DType dt, const LayerNormArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  int grid = 0;
  return dt == DType::F32 ? pick_rows<false, float>(a, &grid, stream)
                          : pick_rows<false, __nv_bfloat16>(a, &grid, stream);
}

cudaError_t launch_layer_norm_bwd(DType dt, const LayerNormArgs& a, float* dw, float* db, cudaStream_t stream) {
  int grid = 0;
  if (a.T > 0) {
    const cudaError_t e = dt == DType::F32 ? pick_rows<true, float>(a, &grid, stream)
                                           : pick_rows<true, __nv_bfloat16>(a, &grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (dw == nullptr && db == nullptr) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((a.D + 31) / 32, 2);
  cfg.blockDim = dim3(32, 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.T > 0 ? 1 : 0;  // not before what another call launched
  const float* part = a.part;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, layer_norm_sum_kernel, part, dw, db, grid, a.D);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rapt
