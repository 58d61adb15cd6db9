// Layer norm of rows of D values, and its gradients (sm_103a):
//   y = w xh + b,  xh = (x - m) r,  m = mean x,  r = (mean (x - m)^2 + eps)^(-1/2)
//   dx = r (g - mean g - xh mean(g xh)),  g = w dy,  dw = sum_rows dy xh,  db = sum_rows dy.
//
// HBM bound: the forward moves 2 tensors, the backward 3, each once. Rows lie and arrive as in the residual norm
// (residual_norm.cuh): a CTA takes a row at a time (8 to 32 lanes take a narrow one), the rows ahead are in
// flight in a ring in shared memory, each thread copies and reads its own columns alone. A row has two reductions:
// its mean first, then the sums over xc = x - m, so that the variance is a sum of squared differences. With the
// mean's own rounding error c = mean xc,
//   var = mean xc^2 - c^2,  xh = (xc - c) r,  sum g xh = r (sum g xc - c sum g):
// a row whose mean is 1e4 times its deviation keeps the bits that its values have. The backward's column sums
// stay in registers over the CTA's rows (fp32); a second small launch adds the CTAs' in a fixed order.
//
// What it costs beside the bytes is instructions: unpacking, five to ten of arithmetic a value, and the reductions,
// which a thread pays once a row. So threads take many columns, and rows that fill them take no checks. The forward of
// 16384 x 2048 bf16: one reduction that carries the next row's sum (x unpacked twice) 39 us with 8 columns a thread, 33
// with 16; two reductions 31; no checks 26. Its backward: 44 us (48 with 16 columns instead of 32), some 6 of it for
// the sum over the CTAs. 4099 x 5121 fp32, backward: 70 us.
#include "residual_norm.cuh"
#include "tc_utils.cuh"

namespace rapt {
namespace {

using namespace rn;

__device__ __forceinline__ float sum4(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float2 add4(Quad a, float2 s) {
  return __fadd2_rn(a.p[1], __fadd2_rn(a.p[0], s));
}
__device__ __forceinline__ Quad add4(Quad a, Quad b) {
  return {{__fadd2_rn(a.p[0], b.p[0]), __fadd2_rn(a.p[1], b.p[1])}};
}

// f + v where there is a column, else zeros.
template <typename C, bool FULL, int NC>
__device__ __forceinline__ void shift(const C& in, Quad (&f)[NC], float v) {
  constexpr int Q = C::kPer / 4;  // quads of a piece
#pragma unroll
  for (int i = 0; i < C::kPieces; ++i) {
    const int e = in.col(i);
    const Quad by = quad(FULL || e < in.D ? v : 0.f);  // pieces behind the row are zeros
#pragma unroll
    for (int q = 0; q < Q; ++q) f[i * Q + q] = add4(f[i * Q + q], by);
    if (e >= in.D || in.whole(i)) continue;
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

// Sums N = 1, 2 or 4 values over the threads of a row: the warps halve the values with the distance, then every
// warp adds the warps' sums in the same order (up to four: every thread by itself). Two calls in turn with buffers
// of their own need one barrier each: a buffer is written again behind the other call's barrier, which follows its
// last read.
template <int N, int MAXT>
__device__ __forceinline__ void sum_row(float (&v)[N], int tpr, float* red) {
  constexpr unsigned kAll = 0xffffffffu;
  constexpr bool kFew = MAXT <= 128;  // red[value][4 warps], else red[warp][value]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5;
  if (warps <= 1) {
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(kAll, v[n], o);
    return;
  }
  float c = v[0];
  if constexpr (N > 1) {
    const bool up = lane & 16;
    float h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      h[i] = (up ? v[i + N / 2] : v[i]) + __shfl_xor_sync(kAll, up ? v[i] : v[i + N / 2], 16);
    c = h[0];
    if constexpr (N == 4) {
      const bool up8 = lane & 8;
      c = (up8 ? h[1] : h[0]) + __shfl_xor_sync(kAll, up8 ? h[0] : h[1], 8);
    }
  }
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) c += __shfl_xor_sync(kAll, c, o);
  const int n0 = lane / (32 / N);
  if (lane % (32 / N) == 0) red[kFew ? n0 * 4 + warp : warp * N + n0] = c;
  __syncthreads();
  if constexpr (kFew) {  // zeros behind the last warp
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float4 q = *reinterpret_cast<const float4*>(red + n * 4);
      v[n] = (q.x + q.y) + (q.z + q.w);
    }
  } else {
    c = 0.f;
    for (int i = lane; i < warps * N; i += 32) c += red[i];  // value lane % N
#pragma unroll
    for (int o = 16; o >= N; o >>= 1) c += __shfl_xor_sync(kAll, c, o);
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = N == 1 ? c : __shfl_sync(kAll, c, n);
  }
}

template <bool BWD, typename T, Rows R, int NC, int STAGES, int MAXT, int MINB, bool FULL>
__global__ void __launch_bounds__(MAXT, MINB) layer_norm_kernel(const LayerNormArgs a, int tpr) {
  using C = Cols<T, R, NC, true, FULL>;
  constexpr int kTensors = BWD ? 2 : 1;  // of a stage: x, dy
  __shared__ __align__(16) float red[2][4 * 32];
  extern __shared__ __align__(16) uint8_t ring[];
  const int tx = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr, D = a.D;
  const float inv_d = 1.f / static_cast<float>(D);
  const long step = static_cast<long>(gridDim.x) * slots, step_off = step * D;
  const long row = static_cast<long>(blockIdx.x) * slots + slot;
  const C in(tx, tpr, D, row);
  // the rows of a warp end together: those past T are zeros and not stored
  const int rows = row < a.T ? static_cast<int>((a.T - 1 - row) / step) + 1 : 0;
  const int turns = static_cast<int>((a.T - 1 - (row - slot)) / step) + 1;
  uint8_t* const mine = ring + threadIdx.x * C::kBytes;
  const uint32_t row_bytes = blockDim.x * C::stride(kTensors);
  long ahead = row * D;  // of the row that is fetched next
  const auto fetch = [&](uint8_t* st, int turn) {
    if (turn < rows) {
      in.fetch(st, 0, static_cast<const T*>(a.x) + ahead);
      if (BWD) in.fetch(st, 1, static_cast<const T*>(a.dy) + ahead);
    } else {
      in.clear(st, 0);
      if (BWD) in.clear(st, 1);
    }
    commit_copies();
    ahead += step_off;
  };
  const auto read = [&](uint8_t* st, int k, Quad (&f)[NC]) { in.read(st, k, static_cast<const T*>(nullptr), f); };
  if (threadIdx.x < 4 * 4) red[0][threadIdx.x] = red[1][threadIdx.x] = 0.f;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) {
    in.clear(mine + s * row_bytes, 0);
    if (BWD) in.clear(mine + s * row_bytes, 1);
    fetch(mine + s * row_bytes, s);
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
  __syncthreads();  // the zeros of `red`
  T* out = static_cast<T*>(a.out) + row * D;
  uint32_t s = 0;  // offset of the row's stage
  for (int i = 0; i < turns; ++i, out += step_off) {
    uint8_t* const st = mine + s;
    s = s + row_bytes == STAGES * row_bytes ? 0 : s + row_bytes;
    wait_copies<STAGES - 1>();
    Quad xc[NC];
    read(st, 0, xc);
    float2 s1 = both(0.f), s2 = s1;
    float m[1];
#pragma unroll
    for (int c = 0; c < NC; ++c) s1 = add4(xc[c], s1);
    m[0] = sum4(s1);
    if (!BWD) fetch(st, i + STAGES);
    sum_row<1, MAXT>(m, tpr, red[0]);
    shift<C, FULL>(in, xc, -m[0] * inv_d);
    s1 = both(0.f);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      s1 = add4(xc[c], s1);
      s2 = dot4(xc[c], xc[c], s2);
    }
    const auto root = [&](float c0, float sq) { return inv_root(fmaxf(fmaf(sq, inv_d, -c0 * c0), 0.f) + a.eps); };
    if constexpr (BWD) {
      float2 g1 = both(0.f), g2 = g1;
      {
        Quad g[NC];
        read(st, 1, g);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          g[c] = g[c] * w[c];
          g1 = add4(g[c], g1);
          g2 = dot4(g[c], xc[c], g2);
        }
      }
      float q[4] = {sum4(s1), sum4(s2), sum4(g1), sum4(g2)};
      sum_row<4, MAXT>(q, tpr, red[1]);
      const float c0 = q[0] * inv_d, r = root(c0, q[1]);
      const float mg = q[2] * inv_d, mgx = r * (q[3] - c0 * q[2]) * inv_d;
      const Quad by = quad(-c0 * r), kx = quad(-mgx * r), kg = quad(-mg * r);
      Quad g[NC];
      read(st, 1, g);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const Quad xh = fma4(xc[c], quad(r), by);
        sw[c] = fma4(g[c], xh, sw[c]);
        sb[c] = add4(g[c], sb[c]);
        xc[c] = fma4(g[c] * w[c], quad(r), fma4(xh, kx, kg));
      }
      fetch(st, i + STAGES);
    } else {
      float q[2] = {sum4(s1), sum4(s2)};
      sum_row<2, MAXT>(q, tpr, red[1]);
      const float c0 = q[0] * inv_d, r = root(c0, q[1]);
      const Quad by = quad(-c0 * r);
#pragma unroll
      for (int c = 0; c < NC; ++c) xc[c] = fma4(fma4(xc[c], quad(r), by), w[c], b[c]);
    }
    in.write(a.out != nullptr && i < rows ? out : nullptr, xc);
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
  constexpr int kAhead = 10;  // loads in flight
  __shared__ float s[32][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* const out = k == 0 ? dw : db;
  float v = 0.f;
  tc::grid_dep_wait();  // the partials of the launch before this one
  if (c < D && out != nullptr) {
    for (int b = threadIdx.y; b < nparts; b += 32 * kAhead) {
      float p[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        p[i] = b + 32 * i < nparts ? part[(static_cast<long>(b + 32 * i) * 2 + k) * D + c] : 0.f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) v += p[i];
    }
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || c >= D || out == nullptr) return;
  float t = 0.f;
#pragma unroll
  for (int q = 0; q < 32; ++q) t += s[q][threadIdx.x];
  out[c] = t;
}

// CTAs of a backward at most: 32 columns a thread take 168 registers and more.
inline int parts(const RowShape& s) { return s.ept == 32 ? 160 * std::max(1, 384 / s.threads) : max_parts(s); }

template <bool BWD, typename T, Rows R, int NC, int STAGES, int MAXT, int MINB, bool FULL = false>
cudaError_t go(const LayerNormArgs& a, const RowShape& s, int* grid, cudaStream_t stream) {
  size_t smem = ring_bytes<T, R, NC>(s, STAGES, BWD ? 2 : 1);
  // the slots' column sums meet where the ring was
  if (BWD && s.tpr <= 32) smem = std::max(smem, static_cast<size_t>(s.threads / s.tpr) * 2 * a.D * 4);
  return launch_rows<layer_norm_kernel<BWD, T, R, NC, STAGES, MAXT, MINB, FULL>>(
      a, s, smem, BWD ? parts(s) : 1 << 30, kMore<T, R> + 1, grid, stream);
}
// Columns a thread. 128 MiB a tensor, us: backward with 32 where the row is 32 times its threads, else 16: bf16
// D = 2048 76 / 83, 4096 80 / 97, 8192 108 / 117. Forward, bf16: 6144 66 with 16, 83 with 24; 8192 72 with 24, 74
// with 16.
inline RowShape shape(int D, int more, bool bwd) {
  const int n = D + more;
  if (bwd && D % 1024 == 0 && D <= 8192) return row_shape(D, 32, more);
  return row_shape(D, n <= 256 ? 8 : n <= (bwd ? 8192 : 6144) ? 16 : 24, more);
}
template <bool BWD, typename T, Rows R>
cudaError_t pick(const LayerNormArgs& a, int* grid, cudaStream_t stream) {
  const RowShape s = shape(a.D, kMore<T, R>, BWD);
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kS = kF32 || BWD ? 3 : 4;
  if (s.ept == 8) return go<BWD, T, R, 2, kS, 256, BWD ? 3 : 4>(a, s, grid, stream);
  if constexpr (BWD && R == Rows::Whole)
    if (s.ept == 32)
      return s.threads <= 128 ? go<BWD, T, R, 8, 3, 128, 2, true>(a, s, grid, stream)
                              : go<BWD, T, R, 8, 3, 256, 1, true>(a, s, grid, stream);
  if (s.ept == 16) {
    if constexpr (R == Rows::Whole)
      if (a.D == 16 * s.tpr && s.threads <= 256)
        return s.threads <= 128 ? go<BWD, T, R, 4, kS, 128, BWD ? 3 : 5, true>(a, s, grid, stream)
                                : go<BWD, T, R, 4, kS, 256, BWD ? 2 : 3, true>(a, s, grid, stream);
    if (s.threads <= 128) return go<BWD, T, R, 4, kS, 128, BWD ? 3 : 5>(a, s, grid, stream);
    if (s.threads <= 256) return go<BWD, T, R, 4, kS, 256, BWD ? 2 : 3>(a, s, grid, stream);
    // a deep ring for one CTA an SM: 5121 columns fp32 70 us, 108 with two stages; two CTAs (spills) 101
    if constexpr (BWD)
      return s.threads <= 384 ? go<BWD, T, R, 4, 4, 384, 1>(a, s, grid, stream)
                              : go<BWD, T, R, 4, kF32 ? 3 : 4, 512, 1>(a, s, grid, stream);
    else
      return go<BWD, T, R, 4, kS, 384, 2>(a, s, grid, stream);  // 5120 bf16 68 us; one CTA an SM 98
  }
  if (!BWD && s.threads <= 352) return go<BWD, T, R, 6, 3, 352, 1>(a, s, grid, stream);
  if (s.threads <= 512) return go<BWD, T, R, 6, 2, 512, 1>(a, s, grid, stream);
  return go<BWD, T, R, 6, BWD && kF32 ? 1 : 2, 704, 1>(a, s, grid, stream);
}
template <bool BWD, typename T>
cudaError_t pick_rows(const LayerNormArgs& a, int* grid, cudaStream_t stream) {
  return whole_rows<T>(a.D) ? pick<BWD, T, Rows::Whole>(a, grid, stream) : pick<BWD, T, Rows::Shifted>(a, grid, stream);
}

}  // namespace

size_t layer_norm_ws_bytes(long T, int D, DType dt) {
  const int vec = dt == DType::F32 ? kVec<float> : kVec<__nv_bfloat16>;
  const RowShape s = shape(D, D % vec == 0 ? 0 : vec - 1, true);
  const long slots = s.threads / s.tpr;
  return static_cast<size_t>(std::min<long>((T + slots - 1) / slots, parts(s))) * 2 * D * 4;
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
