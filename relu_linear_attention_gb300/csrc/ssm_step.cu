// One token of the selective scan for N sequences (sm_103a). Per (sequence, head), with dt the step size:
//   S = exp(dt A) S + dt B x^T  (N x P, in place),   y = (S^T C + D x) silu(z).
//
// A pure stream of the fp32 states: every element is read once and written once by 16-byte accesses, all of a
// thread's loads before its first use, and the columns' sums over the rows meet in shared memory. A column of S
// depends on no other: where sequences and heads are few, a head's columns are spread over CTAs. States of less
// than a CTA's share go several heads to a CTA.
#include "ssm.cuh"

namespace rapt {
namespace {

using namespace ssm;

constexpr int kThreads = 256;

// PC columns of a head's P to a CTA's group of threads: CG column groups of 4, RG row groups, ROWS rows a thread.
template <int N, int PC>
struct Cfg {
  static constexpr int CG = PC / 4;
  static constexpr int RG = kThreads / CG < N ? kThreads / CG : N;
  static constexpr int ROWS = N / RG;
  static constexpr int THREADS = CG * RG;            // of a head's part
  static constexpr int PARTS = kThreads / THREADS;   // heads' parts in a CTA
};

template <typename T, int N, int P, int PC>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(const SsmArgs a, float* S, long units) {
  using C = Cfg<N, PC>;
  __shared__ __align__(16) float red[C::PARTS][C::RG][PC];
  __shared__ __align__(16) float bs[C::PARTS][N], cs[C::PARTS][N], xs[C::PARTS][PC];
  const int part = threadIdx.x / C::THREADS, tid = threadIdx.x % C::THREADS;
  const long unit = static_cast<long>(blockIdx.x) * C::PARTS + part;
  const bool live = unit < units;
  const int slice = static_cast<int>(unit % (P / PC));
  const long nh = unit / (P / PC);
  const int h = static_cast<int>(nh % a.H), g = h / (a.H / a.G), p0 = slice * PC;
  const long n = nh / a.H;
  const int cg = tid % C::CG, rg = tid / C::CG;

  float4 s[C::ROWS];
  float* const Sh = S + nh * (N * P) + p0 + 4 * cg;
  float step = 0.f, keep = 0.f;
  if (live) {
#pragma unroll
    for (int m = 0; m < C::ROWS; ++m)
      s[m] = __ldcs(reinterpret_cast<const float4*>(Sh + (rg + m * C::RG) * P));
    step = step_size(to_f(static_cast<const T*>(a.dt)[n * a.dts + h]), a.dt_bias != nullptr ? a.dt_bias[h] : 0.f,
                     a.softplus);
    keep = expf(step * a.A[h]);
    for (int i = tid; i < N; i += C::THREADS) {
      bs[part][i] = step * to_f(static_cast<const T*>(a.B)[n * a.bs + g * N + i]);
      cs[part][i] = to_f(static_cast<const T*>(a.C)[n * a.cs + g * N + i]);
    }
    for (int i = tid; i < PC; i += C::THREADS) xs[part][i] = to_f(static_cast<const T*>(a.x)[n * a.xs + h * P + p0 + i]);
  }
  __syncthreads();
  if (live) {
    const float4 x = *reinterpret_cast<const float4*>(&xs[part][4 * cg]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < C::ROWS; ++m) {
      const int i = rg + m * C::RG;
      const float b = bs[part][i], c = cs[part][i];
      float4 v = s[m];
      v.x = fmaf(keep, v.x, b * x.x);
      v.y = fmaf(keep, v.y, b * x.y);
      v.z = fmaf(keep, v.z, b * x.z);
      v.w = fmaf(keep, v.w, b * x.w);
      __stcs(reinterpret_cast<float4*>(Sh + i * P), v);
      y.x = fmaf(c, v.x, y.x);
      y.y = fmaf(c, v.y, y.y);
      y.z = fmaf(c, v.z, y.z);
      y.w = fmaf(c, v.w, y.w);
    }
    *reinterpret_cast<float4*>(&red[part][rg][4 * cg]) = y;
  }
  __syncthreads();
  if (!live) return;
  for (int j = tid; j < PC; j += C::THREADS) {
    float y = 0.f;
#pragma unroll
    for (int r = 0; r < C::RG; ++r) y += red[part][r][j];
    if (a.D != nullptr) y = fmaf(a.D[h], xs[part][j], y);
    if (a.z != nullptr) {
      const float z = to_f(static_cast<const T*>(a.z)[n * a.zs + h * P + p0 + j]);
      y *= z * sigmoid_f(z);
    }
    static_cast<T*>(a.out)[nh * P + p0 + j] = from_float<T>(y);
  }
}

template <typename T, int N, int P, int PC>
cudaError_t go(const SsmArgs& a, float* S, cudaStream_t stream) {
  const long units = static_cast<long>(a.docs.n_docs) * a.H * (P / PC);
  const long grid = (units + Cfg<N, PC>::PARTS - 1) / Cfg<N, PC>::PARTS;
  ssm_step_kernel<T, N, P, PC><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a, S, units);
  note_launches(1);
  return cudaGetLastError();
}
template <typename T, int N, int P>
cudaError_t by_part(const SsmArgs& a, float* S, cudaStream_t stream) {
  const long heads = static_cast<long>(a.docs.n_docs) * a.H;
  if constexpr (P >= 64 && N >= 64)
    if (heads < 512) return go<T, N, P, 16>(a, S, stream);
  return go<T, N, P, P>(a, S, stream);
}
template <typename T, int N>
cudaError_t by_p(const SsmArgs& a, float* S, cudaStream_t s) {
  switch (a.P) {
    case 16: return by_part<T, N, 16>(a, S, s);
    case 32: return by_part<T, N, 32>(a, S, s);
    case 64: return by_part<T, N, 64>(a, S, s);
    case 128: return by_part<T, N, 128>(a, S, s);
    default: return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t by_n(const SsmArgs& a, float* S, cudaStream_t s) {
  switch (a.N) {
    case 16: return by_p<T, 16>(a, S, s);
    case 32: return by_p<T, 32>(a, S, s);
    case 64: return by_p<T, 64>(a, S, s);
    case 128: return by_p<T, 128>(a, S, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_ssm_step(DType dt, const SsmArgs& a, float* S, cudaStream_t stream) {
  return dt == DType::F32 ? by_n<float>(a, S, stream) : by_n<__nv_bfloat16>(a, S, stream);
}

}  // namespace rapt
