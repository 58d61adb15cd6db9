// The gated feed-forward of few tokens (decoding): h = act(x w_gate^T) (x w_up^T) for M <= 16 rows, bf16,
// fp32 accumulation, sm_103a.
//
// The weights are read once and decide the time (HBM bound: 4 F K bytes). They are the 16-row operand of
// warp-level bf16 products (mma.sync m16n8k16), eight rows of w_gate above the same eight of w_up, and go
// from memory to registers without a detour: a product sums over k in any order as long as both operands
// agree, so a thread takes the 16 bytes (eight k) that follow each other in its weight row and in its
// token's row, and calls them the fragment's k. One CTA forms eight columns of h for all tokens: F / 8
// small CTAs are all resident at once and spread evenly (16 columns and twice the threads a CTA: 344
// CTAs for 304 places at F = 5504). Its four warps take every fourth 32-deep slice of k, AHEAD slices of
// loads before the products. The warps' sums meet in shared memory and are added in warp order: the same
// bits every time.
#include "activation.cuh"
#include "kernels.h"

namespace rapt {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kCols = 8;    // columns of h that a CTA forms
constexpr int kSlice = 32;  // k of a slice

struct DecodeGluArgs {
  const __nv_bfloat16 *x, *w_gate, *w_up;
  __nv_bfloat16* h;
  int M, F, K;
  Act act;
};

// 16 bytes that are read once: past L1.
__device__ __forceinline__ uint4 load_stream(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT groups of eight tokens; AHEAD slices of weights in registers.
template <int NT, int AHEAD>
__global__ void __launch_bounds__(kThreads) glu_decode_kernel(const DecodeGluArgs a) {
  __shared__ float4 sums[kWarps][NT][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int f0 = blockIdx.x * kCols;  // F is a multiple of eight
  const __nv_bfloat16* gate = a.w_gate + static_cast<long>(f0 + g) * a.K + 8 * t;
  const __nv_bfloat16* up = a.w_up + static_cast<long>(f0 + g) * a.K + 8 * t;
  const int slices = (a.K + kSlice - 1) / kSlice;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 w[AHEAD][2];
  const auto load_w = [&](int slot, int s) {
    const bool in = s * kSlice + 8 * t < a.K;
    w[slot][0] = in ? load_stream(gate + s * kSlice) : zero;
    w[slot][1] = in ? load_stream(up + s * kSlice) : zero;
  };
  float acc[NT][4] = {};
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load_w(i, warp + i * kWarps);
  for (int s0 = warp; s0 < slices; s0 += AHEAD * kWarps) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int s = s0 + i * kWarps, k = s * kSlice + 8 * t;
      uint4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int m = 8 * n + g;
        b[n] = m < a.M && k < a.K ? *reinterpret_cast<const uint4*>(a.x + static_cast<long>(m) * a.K + k) : zero;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(acc[n], w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, b[n].x, b[n].y);
        mma16816(acc[n], w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, b[n].z, b[n].w);
      }
      load_w(i, s + AHEAD * kWarps);
    }
  }
  // accumulators 0, 1 of lane (g, t): g of column f0 + g for tokens 8 n + 2 t, + 1; 2, 3: u of the same
#pragma unroll
  for (int n = 0; n < NT; ++n) sums[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  __syncthreads();
  for (int e = threadIdx.x; e < 32 * NT; e += kThreads) {
    const int n = e >> 5, from = e & 31;
    float4 v = sums[0][n][from];
#pragma unroll
    for (int q = 1; q < kWarps; ++q) {
      const float4 o = sums[q][n][from];
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    const int f = f0 + (from >> 2), m = 8 * n + 2 * (from & 3);
    float av, da;
    if (m < a.M) {
      act_one<false>(a.act, v.x, av, da);
      a.h[static_cast<long>(m) * a.F + f] = __float2bfloat16_rn(av * v.z);
    }
    if (m + 1 < a.M) {
      act_one<false>(a.act, v.y, av, da);
      a.h[static_cast<long>(m + 1) * a.F + f] = __float2bfloat16_rn(av * v.w);
    }
  }
}

template <int NT, int AHEAD>
cudaError_t go(const DecodeGluArgs& a, cudaStream_t stream) {
  glu_decode_kernel<NT, AHEAD><<<a.F / kCols, kThreads, 0, stream>>>(a);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glu_decode(const GluArgs& g, void* h, cudaStream_t stream) {
  DecodeGluArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(g.x);
  a.w_gate = static_cast<const __nv_bfloat16*>(g.w_gate);
  a.w_up = static_cast<const __nv_bfloat16*>(g.w_up);
  a.h = static_cast<__nv_bfloat16*>(h);
  a.M = g.M;
  a.F = g.F;
  a.K = g.K;
  a.act = g.act;
  if (g.M <= 8) return go<1, 4>(a, stream);
  return g.M <= kGluDecodeRows ? go<2, 4>(a, stream) : cudaErrorInvalidValue;
}

}  // namespace rapt
