// Norms before and after a block, fused with its gate and residual scale (sm_103a).
//
// Forward, per row of D values (x the residual stream, y the block's output, z its gate):
//     n = w_post y sg,  sg = (mean y^2 + eps)^(-1/2)      (n = y without a post norm)
//     r = x + s act(z) n
//     h = w_pre r rho,  rho = (mean r^2 + eps)^(-1/2)
// Backward of sum dr . r + sum dh . h, with a = act(z), rh = r rho, yh = y sg, t = w_pre dh:
//     g  = dr + rho (t - rh mean(t rh)),  dx = g,  dw_pre = sum_rows dh rh
//     dz = s n act'(z) g,  ds = sum_rows a n g
//     dn = s a g,  dw_post = sum_rows dn yh,  u = w_post dn,  dy = sg (u - yh mean(u yh))
// where mean(t rh) = rho mean(t r): the two sums over r need no rho, so they share one reduction.
//
// HBM bound: the forward moves 5 tensors, the backward 8, each once; a row lives in registers
// between its reductions (one for y, one for r, one for u). One CTA takes a row (D > 256) or one
// warp does (D <= 256: the reductions are shuffles alone); each thread owns the same columns of
// every row it meets, so the gains stay in registers and the backward's column sums accumulate in
// fp32 registers over the CTA's rows. Those partials go to the workspace, one row per CTA, and a
// second small launch adds them in CTA order: no atomics, the same bits every time. h is formed from
// the unrounded r. All arithmetic is fp32; every output is rounded once.
#include "activation.cuh"
#include "kernels.h"

namespace rapt {
namespace {

// Elements are owned in vectors of VEC (16 bytes, or single elements where rows are not 16-byte
// aligned); vector c of thread tx starts at column (c * TPR + tx) * VEC.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (VEC == 1) {
    f[0] = static_cast<float>(*p);
  } else {
    float v[VEC];
    RowLoad<T, VEC>::run(p, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = v[i];
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (VEC == 1) {
    *p = from_float<T>(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    store4(p, f[0], f[1], f[2], f[3]);
  } else {
    uint4 w;
    __nv_bfloat162 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w.x = *reinterpret_cast<uint32_t*>(&b[0]);
    w.y = *reinterpret_cast<uint32_t*>(&b[1]);
    w.z = *reinterpret_cast<uint32_t*>(&b[2]);
    w.w = *reinterpret_cast<uint32_t*>(&b[3]);
    *reinterpret_cast<uint4*>(p) = w;
  }
}

// A thread's columns of one row (or of a gain vector) as floats, `fill` past the end.
template <typename T, int VEC, int EPT>
__device__ __forceinline__ void load_cols(const T* row, int tx, int tpr, int D, float fill, float (&f)[EPT]) {
#pragma unroll
  for (int c = 0; c < EPT / VEC; ++c) {
    const int e = (c * tpr + tx) * VEC;
    if (e < D) {
      load_vec<T, VEC>(row + e, f + c * VEC);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[c * VEC + i] = fill;
    }
  }
}
template <typename T, int VEC, int EPT>
__device__ __forceinline__ void store_cols(T* row, int tx, int tpr, int D, const float (&f)[EPT]) {
#pragma unroll
  for (int c = 0; c < EPT / VEC; ++c) {
    const int e = (c * tpr + tx) * VEC;
    if (e < D) store_vec<T, VEC>(row + e, f + c * VEC);
  }
}
// fp32 columns of a gain vector: 1 where there is none, 0 past the end.
template <int VEC, int EPT>
__device__ __forceinline__ void load_gain(const float* w, int tx, int tpr, int D, float (&f)[EPT]) {
#pragma unroll
  for (int c = 0; c < EPT / VEC; ++c) {
    const int e = (c * tpr + tx) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[c * VEC + i] = e < D ? (w != nullptr ? w[e + i] : 1.f) : 0.f;
  }
}

// fp32 column sums to a partial row.
template <int VEC, int EPT>
__device__ __forceinline__ void store_sums(float* row, int tx, int tpr, int D, const float (&f)[EPT]) {
#pragma unroll
  for (int c = 0; c < EPT / VEC; ++c) {
    const int e = (c * tpr + tx) * VEC;
    if (e >= D) continue;
    if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        store4(row + e + i, f[c * VEC + i], f[c * VEC + i + 1], f[c * VEC + i + 2], f[c * VEC + i + 3]);
    } else {
      row[e] = f[c * VEC];
    }
  }
}

// Sums N values over the threads of a row. A row of one warp uses shuffles alone; a row of a whole
// CTA adds the warps' sums from `red` (two alternating halves, so one barrier per call suffices:
// a half is rewritten two calls later, after a barrier that follows its last read).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int warps, float (*red)[2][32], int& half) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red[half][n][warp] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float s = lane < warps ? red[half][n][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    v[n] = s;
  }
  half ^= 1;
}

template <typename T, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_fwd_kernel(const ResidualNormArgs a, int tpr) {
  __shared__ float red[2][2][32];
  int half = 0;
  const int tx = threadIdx.x % tpr, rows_per_cta = blockDim.x / tpr, warps = tpr >> 5;
  const float inv_d = 1.f / static_cast<float>(a.D);
  float wpost[EPT], sc[EPT], wpre[EPT];
  load_gain<VEC, EPT>(a.w_post, tx, tpr, a.D, wpost);
  load_gain<VEC, EPT>(a.scale, tx, tpr, a.D, sc);
  load_gain<VEC, EPT>(a.w_pre, tx, tpr, a.D, wpre);
  const long step = static_cast<long>(gridDim.x) * rows_per_cta;
  for (long row = static_cast<long>(blockIdx.x) * rows_per_cta + threadIdx.x / tpr; row < a.T; row += step) {
    const long off = row * a.D;
    float r[EPT];
    load_cols<T, VEC, EPT>(static_cast<const T*>(a.x) + off, tx, tpr, a.D, 0.f, r);
    if (a.y != nullptr) {
      float n[EPT], z[EPT];
      load_cols<T, VEC, EPT>(static_cast<const T*>(a.y) + off, tx, tpr, a.D, 0.f, n);
      if (a.gate != nullptr) load_cols<T, VEC, EPT>(static_cast<const T*>(a.gate) + off, tx, tpr, a.D, 0.f, z);
      if (a.w_post != nullptr) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < EPT; ++i) s[0] = fmaf(n[i], n[i], s[0]);
        row_sum<1>(s, warps, red, half);
        const float sg = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < EPT; ++i) n[i] *= sg * wpost[i];
      }
      if (a.gate != nullptr) {
        float g[EPT];
        act_vec<EPT, false>(a.act, z, g, z);
#pragma unroll
        for (int i = 0; i < EPT; ++i) n[i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i) r[i] = fmaf(sc[i], n[i], r[i]);
    }
    if (a.r != nullptr) store_cols<T, VEC, EPT>(static_cast<T*>(a.r) + off, tx, tpr, a.D, r);
    if (a.h != nullptr) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < EPT; ++i) s[0] = fmaf(r[i], r[i], s[0]);
      row_sum<1>(s, warps, red, half);
      const float rho = rsqrtf(fmaf(s[0], inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < EPT; ++i) r[i] *= rho * wpre[i];
      store_cols<T, VEC, EPT>(static_cast<T*>(a.h) + off, tx, tpr, a.D, r);
    }
  }
}

// Partial column sums of CTA b at part[(b * 3 + k) * D + column], k = 0: dw_post, 1: dscale, 2: dw_pre.
template <typename T, int VEC, int EPT, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_bwd_kernel(const ResidualNormArgs a, int tpr) {
  __shared__ float red[2][2][32];
  extern __shared__ float s_part[];  // rows per CTA > 1: the warps' partials, [rows][3][D]
  int half = 0;
  const int tx = threadIdx.x % tpr, slot = threadIdx.x / tpr, rows_per_cta = blockDim.x / tpr, warps = tpr >> 5;
  const float inv_d = 1.f / static_cast<float>(a.D);
  float wpost[EPT], sc[EPT], wpre[EPT], gpost[EPT], gsc[EPT], gpre[EPT];
  load_gain<VEC, EPT>(a.w_post, tx, tpr, a.D, wpost);
  load_gain<VEC, EPT>(a.scale, tx, tpr, a.D, sc);
  load_gain<VEC, EPT>(a.w_pre, tx, tpr, a.D, wpre);
#pragma unroll
  for (int i = 0; i < EPT; ++i) gpost[i] = gsc[i] = gpre[i] = 0.f;
  const long step = static_cast<long>(gridDim.x) * rows_per_cta;
  for (long row = static_cast<long>(blockIdx.x) * rows_per_cta + slot; row < a.T; row += step) {
    const long off = row * a.D;
    float g[EPT], y[EPT], an[EPT], dzn[EPT], sg = 1.f;  // an = act(z) n, dzn = act'(z) n
#pragma unroll
    for (int i = 0; i < EPT; ++i) g[i] = y[i] = an[i] = dzn[i] = 0.f;
    if (a.dr != nullptr) load_cols<T, VEC, EPT>(static_cast<const T*>(a.dr) + off, tx, tpr, a.D, 0.f, g);
    float av[EPT];  // act(z)
#pragma unroll
    for (int i = 0; i < EPT; ++i) av[i] = 1.f;
    float t[EPT], r[EPT];
    if (a.dh != nullptr) {
      load_cols<T, VEC, EPT>(static_cast<const T*>(a.dh) + off, tx, tpr, a.D, 0.f, t);
      load_cols<T, VEC, EPT>(static_cast<const T*>(a.x) + off, tx, tpr, a.D, 0.f, r);
    }
    if (a.y != nullptr) {
      float z[EPT];
      load_cols<T, VEC, EPT>(static_cast<const T*>(a.y) + off, tx, tpr, a.D, 0.f, y);
      if (a.gate != nullptr) load_cols<T, VEC, EPT>(static_cast<const T*>(a.gate) + off, tx, tpr, a.D, 0.f, z);
      if (a.w_post != nullptr) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < EPT; ++i) s[0] = fmaf(y[i], y[i], s[0]);
        row_sum<1>(s, warps, red, half);
        sg = rsqrtf(fmaf(s[0], inv_d, a.eps));
      }
      if (a.gate != nullptr) {
        act_vec<EPT, true>(a.act, z, av, dzn);
      }
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const float n = y[i] * sg * wpost[i];
        an[i] = av[i] * n;
        dzn[i] *= n;
      }
    }
    if (a.dh != nullptr) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        r[i] = fmaf(sc[i], an[i], r[i]);
        s[0] = fmaf(r[i], r[i], s[0]);
        s[1] = fmaf(t[i] * wpre[i], r[i], s[1]);
      }
      row_sum<2>(s, warps, red, half);
      const float rho = rsqrtf(fmaf(s[0], inv_d, a.eps));
      const float c = rho * s[1] * inv_d;  // mean(t rh)
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const float rh = r[i] * rho;
        gpre[i] = fmaf(t[i], rh, gpre[i]);
        g[i] = fmaf(rho, fmaf(-rh, c, t[i] * wpre[i]), g[i]);
      }
    }
    if (a.dx != nullptr) store_cols<T, VEC, EPT>(static_cast<T*>(a.dx) + off, tx, tpr, a.D, g);
    if (a.y != nullptr) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        gsc[i] = fmaf(an[i], g[i], gsc[i]);
        g[i] *= sc[i];
        dzn[i] *= g[i];
        g[i] *= av[i];  // dn
      }
      if (a.dgate != nullptr) store_cols<T, VEC, EPT>(static_cast<T*>(a.dgate) + off, tx, tpr, a.D, dzn);
      if (a.w_post != nullptr) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const float yh = y[i] * sg;
          gpost[i] = fmaf(g[i], yh, gpost[i]);
          y[i] = yh;
          g[i] *= wpost[i];
          s[0] = fmaf(g[i], yh, s[0]);
        }
        row_sum<1>(s, warps, red, half);
        const float c = s[0] * inv_d;
#pragma unroll
        for (int i = 0; i < EPT; ++i) g[i] = sg * fmaf(-y[i], c, g[i]);
      }
      if (a.dy != nullptr) store_cols<T, VEC, EPT>(static_cast<T*>(a.dy) + off, tx, tpr, a.D, g);
    }
  }
  if (a.part == nullptr) return;
  float* out = a.part + static_cast<long>(blockIdx.x) * 3 * a.D;
  if (rows_per_cta == 1) {
    store_sums<VEC, EPT>(out, tx, tpr, a.D, gpost);
    store_sums<VEC, EPT>(out + a.D, tx, tpr, a.D, gsc);
    store_sums<VEC, EPT>(out + 2 * a.D, tx, tpr, a.D, gpre);
    return;
  }
  float* mine = s_part + slot * 3 * a.D;
  store_sums<VEC, EPT>(mine, tx, tpr, a.D, gpost);
  store_sums<VEC, EPT>(mine + a.D, tx, tpr, a.D, gsc);
  store_sums<VEC, EPT>(mine + 2 * a.D, tx, tpr, a.D, gpre);
  __syncthreads();
  for (int e = threadIdx.x; e < 3 * a.D; e += blockDim.x) {
    float v = 0.f;
    for (int q = 0; q < rows_per_cta; ++q) v += s_part[q * 3 * a.D + e];
    out[e] = v;
  }
}

// The gain gradients: the CTAs' partial sums added in a fixed order. blockIdx.y picks the vector,
// 32 x 32 threads take 32 columns; thread (c, q) adds partials q, q + 32, ..., then the 32 sums of a
// column are added in order of q. No partials (T = 0) gives zeros.
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(const float* part, int nparts, int D, float* dw_post,
                                                                 float* dscale, float* dw_pre) {
  __shared__ float s[32][33];
  const int k = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* out = k == 0 ? dw_post : (k == 1 ? dscale : dw_pre);
  if (out == nullptr) return;
  float v = 0.f;
  if (c < D) {
#pragma unroll 8
    for (int b = threadIdx.y; b < nparts; b += 32) v += part[(static_cast<long>(b) * 3 + k) * D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 32; ++q) t += s[q][threadIdx.x];
    out[c] = t;
  }
}

// Columns per thread (EPT) and threads per row (a multiple of 32). Eight columns a thread keep the
// forward at 64 registers up to D = 8192 and the backward at 128 up to D = 4096; wider rows take
// sixteen.
struct RowShape {
  int ept, tpr, rows;  // rows per CTA
};
RowShape row_shape(int D, bool bwd) {
  RowShape s;
  s.ept = D <= (bwd ? 4096 : 8192) ? 8 : 16;
  s.tpr = ((D + s.ept - 1) / s.ept + 31) / 32 * 32;
  s.rows = s.tpr == 32 ? 8 : 1;
  return s;
}
// CTAs of a backward launch at most (its registers hold an SM to 1024 threads): the workspace's rows
// of partial sums.
int max_parts(const RowShape& s) { return 160 * (1024 / (s.tpr * s.rows)); }
size_t bwd_smem(const RowShape& s, int D) { return s.rows > 1 ? static_cast<size_t>(s.rows) * 3 * D * 4 : 0; }

// CTAs of a persistent launch: all that fit on the GPU at once, and no more than there are rows.
template <typename K>
cudaError_t row_grid(K kernel, const RowShape& s, long T, size_t smem, int* grid) {
  const long ctas = (T + s.rows - 1) / s.rows;
  int per_sm = 0, sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  if (ctas <= sms) {
    *grid = static_cast<int>(ctas);
    return cudaSuccess;
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.tpr * s.rows, smem);
  if (e != cudaSuccess) return e;
  const long fit = static_cast<long>(sms) * (per_sm > 0 ? per_sm : 1);
  *grid = static_cast<int>(ctas < fit ? ctas : fit);
  return cudaSuccess;
}

template <typename T, int VEC, int EPT, int MAXT>
cudaError_t go_fwd(const ResidualNormArgs& a, const RowShape& s, cudaStream_t stream) {
  const auto kernel = residual_norm_fwd_kernel<T, VEC, EPT, MAXT>;
  int grid = 0;
  const cudaError_t e = row_grid(kernel, s, a.T, 0, &grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, s.tpr * s.rows, 0, stream>>>(a, s.tpr);
  note_launches(1);
  return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t pick_fwd(const ResidualNormArgs& a, cudaStream_t stream) {
  const RowShape s = row_shape(a.D, false);
  if (s.ept == 16) return go_fwd<T, VEC, 16, 1024>(a, s, stream);
  if (s.tpr <= 256) return go_fwd<T, VEC, 8, 256>(a, s, stream);
  if (s.tpr <= 512) return go_fwd<T, VEC, 8, 512>(a, s, stream);
  return go_fwd<T, VEC, 8, 1024>(a, s, stream);
}

template <typename T, int VEC, int EPT, int MAXT>
cudaError_t go_bwd(ResidualNormArgs a, const RowShape& s, int* grid, cudaStream_t stream) {
  const auto kernel = residual_norm_bwd_kernel<T, VEC, EPT, MAXT>;
  const size_t smem = bwd_smem(s, a.D);
  const cudaError_t e = row_grid(kernel, s, a.T, smem, grid);
  if (e != cudaSuccess) return e;
  if (*grid > max_parts(s)) *grid = max_parts(s);
  kernel<<<*grid, s.tpr * s.rows, smem, stream>>>(a, s.tpr);
  note_launches(1);
  return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t pick_bwd(const ResidualNormArgs& a, int* grid, cudaStream_t stream) {
  const RowShape s = row_shape(a.D, true);
  if (s.ept == 16)
    return s.tpr <= 512 ? go_bwd<T, VEC, 16, 512>(a, s, grid, stream) : go_bwd<T, VEC, 16, 1024>(a, s, grid, stream);
  return s.tpr <= 256 ? go_bwd<T, VEC, 8, 256>(a, s, grid, stream) : go_bwd<T, VEC, 8, 512>(a, s, grid, stream);
}

}  // namespace

size_t residual_norm_ws_bytes(long T, int D) {
  const RowShape s = row_shape(D, true);
  const long ctas = (T + s.rows - 1) / s.rows;
  return static_cast<size_t>(ctas < max_parts(s) ? ctas : max_parts(s)) * 3 * D * 4;
}

cudaError_t launch_residual_norm_fwd(DType dt, const ResidualNormArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  if (dt == DType::BF16)
    return a.D % 8 == 0 ? pick_fwd<__nv_bfloat16, 8>(a, stream) : pick_fwd<__nv_bfloat16, 1>(a, stream);
  return a.D % 4 == 0 ? pick_fwd<float, 4>(a, stream) : pick_fwd<float, 1>(a, stream);
}

cudaError_t launch_residual_norm_bwd(DType dt, const ResidualNormArgs& a, float* dw_post, float* dscale,
                                     float* dw_pre, cudaStream_t stream) {
  int grid = 0;
  if (a.T > 0) {
    cudaError_t e;
    if (dt == DType::BF16)
      e = a.D % 8 == 0 ? pick_bwd<__nv_bfloat16, 8>(a, &grid, stream) : pick_bwd<__nv_bfloat16, 1>(a, &grid, stream);
    else
      e = a.D % 4 == 0 ? pick_bwd<float, 4>(a, &grid, stream) : pick_bwd<float, 1>(a, &grid, stream);
    if (e != cudaSuccess) return e;
  }
  if (dw_post == nullptr && dscale == nullptr && dw_pre == nullptr) return cudaSuccess;
  residual_norm_sum_kernel<<<dim3((a.D + 31) / 32, 3), dim3(32, 32), 0, stream>>>(a.part, grid, a.D, dw_post, dscale,
                                                                                 dw_pre);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace rapt
