// The selective scan as its recurrence, in fp32 on the CUDA cores (sm_103a): fp32 inputs, and heads or states too
// small for the tensor cores' tiles.
//   S_t = exp(dt_t A) S_{t-1} + dt_t B_t x_t^T,   y_t = (S_t^T C_t + D x_t) silu(z_t).
//
// Three multiply-adds a state element and token, and a chain within each token (B and C from shared memory, the sums
// over lanes) that the few warps whose states fit do not hide: 4 x 4096 tokens x 64 heads of 64, N = 128, fp32: 1.96 ms
// (issue slots 43 % busy; the bytes alone 123 us); N = 16 in bf16: 515 us (52 %; 60 us). S stays in registers: a warp
// owns CW columns of a head's state, TN lanes along its N rows and TC along the columns, each lane NE x NC elements, so
// that a value of B or C read from shared memory serves NC columns. The TN partial sums of y meet by halving exchanges.
// Tokens come in stages of kTokens through a ring of cp.async copies; bf16 is widened once per stage for all warps. A
// document cut into segments (few heads, long documents) is first run without reading S out, for the increments of all
// its segments but the last; each segment then starts from S0 and the increments before it, in order.
#include <algorithm>

#include "ssm.cuh"
#include "tc_utils.cuh"

namespace rapt {
namespace {

using namespace ssm;

constexpr int kTokens = 16;  // of a stage
constexpr int kStages = 3;

template <typename T, int N, int P>
struct Cfg {
  static constexpr int TN = N <= 32 ? 4 : 8, NE = N / TN, TC = 32 / TN;
  static constexpr int NC = TC * 4 <= P ? 4 : 2;
  static constexpr int CW = TC * NC, WARPS = P / CW, THREADS = 32 * WARPS;
  static constexpr bool kWiden = sizeof(T) == 2;
  // bytes of a raw stage: B and C rows of N, x and z rows of P
  static constexpr int ROW = (2 * N + 2 * P) * static_cast<int>(sizeof(T));
  static constexpr int STAGE = kTokens * ROW;
  static constexpr int WORK = kWiden ? kTokens * (2 * N + P) * 4 : 0;  // widened B, C, x
  static constexpr int SMEM = kStages * STAGE + WORK + kTokens * P * 4 /* y */ + 2 * kTokens * 4;
};

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

template <typename T, int N, int P, bool READ>
__global__ void __launch_bounds__(Cfg<T, N, P>::THREADS) ssm_simt_kernel(const SsmArgs a) {
  using C = Cfg<T, N, P>;
  constexpr int TN = C::TN, NE = C::NE, NC = C::NC, V = kVec<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* const work = reinterpret_cast<float*>(smem + kStages * C::STAGE);
  float* const ys = reinterpret_cast<float*>(smem + kStages * C::STAGE + C::WORK);
  float* const keeps = ys + kTokens * P;  // exp(dt A), then dt
  float* const steps = keeps + kTokens;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nseg = READ ? a.nseg : a.nseg - 1;  // the last segment's increment is no one's start
  const int seg = static_cast<int>(blockIdx.x % nseg);
  const long dh = blockIdx.x / nseg;
  const int doc = static_cast<int>(dh / a.H), h = static_cast<int>(dh % a.H), g = h / (a.H / a.G);
  long row0;
  int n;
  const bool good = doc_rows(a.docs, doc, row0, n);
  if (READ && !good && seg == 0 && h == 0 && tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, 1u);
  const int segs = n > 0 ? (n + a.seg_len - 1) / a.seg_len : 1;
  if (seg >= (READ ? segs : segs - 1) || (READ && !good)) {
    if (READ) end_behind_records(a);
    return;
  }
  const int t0 = seg * a.seg_len, len = min(a.seg_len, n - t0);  // 0: an empty document
  const long start = row0;
  row0 += t0;

  const int tn = lane % TN, tc = lane / TN, col = warp * C::CW + tc * NC;
  float s[NE][NC];
#pragma unroll
  for (int i = 0; i < NE; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) s[i][c] = 0.f;
  // row of S of this lane's element i: four consecutive ones, then those of the other lanes
  const auto row_of = [&](int i) { return ((i / 4) * TN + tn) * 4 + i % 4; };
  const T* const xg = static_cast<const T*>(a.x) + row0 * a.xs + static_cast<long>(h) * P;
  const T* const bg = static_cast<const T*>(a.B) + row0 * a.bs + static_cast<long>(g) * N;
  const T* const cg = static_cast<const T*>(a.C) + row0 * a.cs + static_cast<long>(g) * N;
  const T* const zg = a.z != nullptr ? static_cast<const T*>(a.z) + row0 * a.zs + static_cast<long>(h) * P : nullptr;
  const T* const dtg = static_cast<const T*>(a.dt) + row0 * a.dts + h;
  // a raw stage: [kTokens][N] of B, of C, [kTokens][P] of x, of z
  const auto fetch = [&](int t) {
    uint8_t* const st = smem + (t / kTokens) % kStages * C::STAGE;
    T* const rb = reinterpret_cast<T*>(st);
    T* const rc = rb + kTokens * N;
    T* const rx = rc + kTokens * N;
    T* const rz = rx + kTokens * P;
    const int m = min(kTokens, len - t);
    for (int i = tid; i < m * (N / V); i += C::THREADS) {
      const int r = i / (N / V), e = i % (N / V) * V;
      copy16(rb + r * N + e, bg + (t + r) * a.bs + e);
      if (READ) copy16(rc + r * N + e, cg + (t + r) * a.cs + e);
    }
    for (int i = tid; i < m * (P / V); i += C::THREADS) {
      const int r = i / (P / V), e = i % (P / V) * V;
      copy16(rx + r * P + e, xg + (t + r) * a.xs + e);
      if (READ && zg != nullptr) copy16(rz + r * P + e, zg + (t + r) * a.zs + e);
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (i * kTokens < len) fetch(i * kTokens);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  constexpr long kRec = N * P + kSsmRecTail;
  if (READ) {
    if (a.nseg > 1) tc::grid_dep_wait();  // a segment's record holds the state at its end by now
    const float* const from = seg > 0           ? a.ws + record(a, doc, start, seg - 1, h) * kRec
                              : a.S0 != nullptr ? a.S0 + dh * (N * P)
                                                : nullptr;
    if (from != nullptr) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) s[i][c] = from[row_of(i) * P + col + c];
    }
  }
  const float bias = a.dt_bias != nullptr ? a.dt_bias[h] : 0.f, A = a.A[h];
  const float skip = READ && a.D != nullptr ? a.D[h] : 0.f;
  float raw = tid < min(kTokens, len) ? to_f(dtg[tid * a.dts]) : 0.f;
  float total = 1.f;  // the decay over the segment

  for (int t = 0; t < len; t += kTokens) {
    const int m = min(kTokens, len - t);
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    if (tid < m) {
      const float step = step_size(raw, bias, a.softplus);
      steps[tid] = step;
      keeps[tid] = expf(step * A);
    }
    if (t + kTokens + tid < len && tid < kTokens) raw = to_f(dtg[(t + kTokens + tid) * a.dts]);
    __syncthreads();  // the stage has arrived for all, the last one's y has been taken
    uint8_t* const st = smem + (t / kTokens) % kStages * C::STAGE;
    const T* const rx = reinterpret_cast<const T*>(st) + 2 * kTokens * N;
    const float *b = reinterpret_cast<const float*>(st), *c = b + kTokens * N, *x = c + kTokens * N;
    if constexpr (C::kWiden) {
      for (int i = tid; i < kTokens * (2 * N + P) / V; i += C::THREADS) {
        float f[V];
        widen<T>(reinterpret_cast<const uint4*>(st)[i], f);
#pragma unroll
        for (int v = 0; v < V; v += 4)
          *reinterpret_cast<float4*>(work + i * V + v) = make_float4(f[v], f[v + 1], f[v + 2], f[v + 3]);
      }
      b = work, c = b + kTokens * N, x = c + kTokens * N;
      __syncthreads();
    }
    if (t + (kStages - 1) * kTokens < len) fetch(t + (kStages - 1) * kTokens);
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll 2
    for (int r = 0; r < m; ++r) {
      const float keep = keeps[r], step = steps[r];
      float xd[NC], y[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        xd[k] = step * x[r * P + col + k];
        y[k] = 0.f;
      }
      total *= keep;
#pragma unroll
      for (int q = 0; q < NE / 4; ++q) {
        const float4 b4 = *reinterpret_cast<const float4*>(b + r * N + (q * TN + tn) * 4);
        const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
        float4 c4;
        if (READ) c4 = *reinterpret_cast<const float4*>(c + r * N + (q * TN + tn) * 4);
        const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < NC; k += 2) {  // two columns an instruction
            float2 v = make_float2(s[4 * q + e][k], s[4 * q + e][k + 1]);
            v = __ffma2_rn(make_float2(keep, keep), v,
                           __fmul2_rn(make_float2(bb[e], bb[e]), make_float2(xd[k], xd[k + 1])));
            s[4 * q + e][k] = v.x;
            s[4 * q + e][k + 1] = v.y;
            if (READ) {
              const float2 w = __ffma2_rn(make_float2(cc[e], cc[e]), v, make_float2(y[k], y[k + 1]));
              y[k] = w.x;
              y[k + 1] = w.y;
            }
          }
      }
      if (READ) {  // lanes with one tc add up: each keeps half of its columns as long as it has several
        float v[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) v[k] = y[k];
        int at = 0;
        int o = TN / 2;
#pragma unroll
        for (int w = NC / 2; w >= 1; w /= 2, o /= 2) {
          const bool up = lane & o;
#pragma unroll
          for (int k = 0; k < w; ++k) {
            const float give = up ? v[k] : v[k + w], have = up ? v[k + w] : v[k];
            v[k] = have + __shfl_xor_sync(0xffffffffu, give, o);
          }
          at += up ? w : 0;
        }
        for (; o >= 1; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        ys[r * P + col + at] = v[0];  // (lanes with the same column write the same value)
      }
    }
    if (READ) {
      __syncthreads();
      const T* const rz = rx + kTokens * P;
      T* const out = static_cast<T*>(a.out) + ((row0 + t) * a.H + h) * P;
      for (int i = tid; i < m * (P / V); i += C::THREADS) {
        const int r = i / (P / V), e = i % (P / V) * V;
        float xv[V], zv[V], f[V];
        widen<T>(*reinterpret_cast<const uint4*>(rx + r * P + e), xv);
        if (zg != nullptr) widen<T>(*reinterpret_cast<const uint4*>(rz + r * P + e), zv);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          f[v] = fmaf(skip, xv[v], ys[r * P + e + v]);
          if (zg != nullptr) f[v] *= zv[v] * sigmoid_f(zv[v]);
        }
        *reinterpret_cast<uint4*>(out + static_cast<long>(r) * a.H * P + e) = narrow<T>(f);
      }
    } else {
      __syncthreads();  // before the next stage's step sizes
    }
  }
  float* dst = nullptr;
  if (!READ) {
    dst = a.ws + record(a, doc, start, seg, h) * kRec;
    if (tid == 0) dst[N * P] = total;
  } else if (seg == segs - 1 && a.S_final != nullptr) {
    dst = a.S_final + dh * (N * P);
  }
  if (dst != nullptr) {
#pragma unroll
    for (int i = 0; i < NE; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) dst[row_of(i) * P + col + c] = s[i][c];
  }
}

// The records of a (document, head)'s segments, increments and decays, become the states at the segments' ends:
// h_j = decay_j h_{j-1} + increment_j from S0. A thread takes four values through the segments, eight records' loads
// ahead of their use; the number of segments is the document's own.
__global__ void __launch_bounds__(256) ssm_prefix_kernel(const SsmArgs a, int np4) {
  tc::grid_launch_dependents();
  const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
  const long dh = i / np4;
  const int e = static_cast<int>(i % np4);
  if (dh >= static_cast<long>(a.docs.n_docs) * a.H) return;
  const int doc = static_cast<int>(dh / a.H);
  long row0;
  int n;
  doc_rows(a.docs, doc, row0, n);
  const int segs = n > 0 ? (n + a.seg_len - 1) / a.seg_len : 1;
  const long rec = 4L * np4 + kSsmRecTail, step = rec * a.H;  // from a segment's to the next one's
  float* const base = a.ws + record(a, doc, row0, 0, static_cast<int>(dh % a.H)) * rec;
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.S0 != nullptr) h = reinterpret_cast<const float4*>(a.S0)[dh * np4 + e];
  tc::grid_dep_wait();
  constexpr int kAhead = 8;
  for (int j0 = 0; j0 < segs - 1; j0 += kAhead) {
    float4 inc[kAhead];
    float keep[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j >= segs - 1) break;
      inc[j] = __ldcg(reinterpret_cast<const float4*>(base + (j0 + j) * step) + e);
      keep[j] = __ldcg(base + (j0 + j) * step + 4 * np4);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j >= segs - 1) break;
      h.x = fmaf(keep[j], h.x, inc[j].x);
      h.y = fmaf(keep[j], h.y, inc[j].y);
      h.z = fmaf(keep[j], h.z, inc[j].z);
      h.w = fmaf(keep[j], h.w, inc[j].w);
      __stcg(reinterpret_cast<float4*>(base + (j0 + j) * step) + e, h);
    }
  }
}

template <typename T, int N, int P, bool READ>
cudaError_t go(const SsmArgs& a, cudaStream_t stream) {
  using C = Cfg<T, N, P>;
  const long grid = static_cast<long>(a.docs.n_docs) * a.H * (READ ? a.nseg : a.nseg - 1);
  if (grid == 0) return cudaSuccess;
  if (C::SMEM > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(ssm_simt_kernel<T, N, P, READ>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = READ && a.nseg > 1 ? 1 : 0;  // behind the prefix kernel alone: inputs are read before it ends
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ssm_simt_kernel<T, N, P, READ>, a);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, int N, int P>
cudaError_t both(const SsmArgs& a, cudaStream_t stream) {
  if (a.nseg > 1) {
    cudaError_t e = go<T, N, P, false>(a, stream);
    if (e == cudaSuccess) e = launch_ssm_prefix(a, stream);
    if (e != cudaSuccess) return e;
  }
  return go<T, N, P, true>(a, stream);
}
template <typename T, int N>
cudaError_t by_p(const SsmArgs& a, cudaStream_t s) {
  switch (a.P) {
    case 16: return both<T, N, 16>(a, s);
    case 32: return both<T, N, 32>(a, s);
    case 64: return both<T, N, 64>(a, s);
    case 128: return both<T, N, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t by_n(const SsmArgs& a, cudaStream_t s) {
  switch (a.N) {
    case 16: return by_p<T, 16>(a, s);
    case 32: return by_p<T, 32>(a, s);
    case 64: return by_p<T, 64>(a, s);
    case 128: return by_p<T, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// Segments: as many as give the GPU about 16 warps an SM, of about 96 tokens at least (what a document leaves is spread:
// never below 64). 3 x 1531 tokens x 24 heads of 32, N = 16, fp32: 39 us; 68 with 256 tokens, whose few warps wait for
// their own arithmetic, 43 with 64, whose CTAs no longer fit the SMs at once. Measured at that size alone.
SsmPlan ssm_plan_simt(const SsmArgs& a) {
  const int warps = std::max(1, a.P / (a.N <= 32 ? (a.P >= 32 ? 32 : 16) : 16));
  const long units = static_cast<long>(a.docs.n_docs) * a.H, longest = a.docs.max_seqlen;
  const long want = 152L * 16 / warps;
  long nseg = std::min<long>({(want + units - 1) / units, (longest + 95) / 96, 64});
  nseg = std::max<long>(nseg, 1);
  SsmPlan p{};
  p.seg_len = static_cast<int>((longest + nseg - 1) / nseg + kTokens - 1) / kTokens * kTokens;
  p.seg_len = std::max(p.seg_len, kTokens);
  p.nseg = static_cast<int>(std::max<long>((longest + p.seg_len - 1) / p.seg_len, 1));
  p.ws_bytes = static_cast<size_t>(ssm_records(a, p.nseg, p.seg_len)) * a.H *
               (static_cast<size_t>(a.N) * a.P + kSsmRecTail) * 4;
  return p;
}

cudaError_t launch_ssm_prefix(const SsmArgs& a, cudaStream_t stream) {
  const int np4 = a.N * a.P / 4;
  const long items = static_cast<long>(a.docs.n_docs) * a.H * np4;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((items + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;  // behind the increments' kernel, which reads nothing that this one writes
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ssm_prefix_kernel, a, np4);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_ssm_simt(DType dt, const SsmArgs& a, cudaStream_t stream) {
  return dt == DType::F32 ? by_n<float>(a, stream) : by_n<__nv_bfloat16>(a, stream);
}

}  // namespace rapt
