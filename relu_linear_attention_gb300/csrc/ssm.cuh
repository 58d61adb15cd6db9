// Device helpers of the selective state space operators (sm_103a): document bounds, step sizes, elements.
#pragma once

#include "kernels.h"
#include "tc_utils.cuh"

namespace rapt {
namespace ssm {

// Rows [row0, row0 + n) of document `doc`; false (and no rows) where cu_seqlens is malformed there.
__device__ __forceinline__ bool doc_rows(const Docs& d, int doc, long& row0, int& n) {
  if (d.cu_seqlens == nullptr) {
    row0 = static_cast<long>(doc) * d.doc_len;
    n = d.doc_len;
    return true;
  }
  const int s = d.cu_seqlens[doc], e = d.cu_seqlens[doc + 1], prev = doc > 0 ? d.cu_seqlens[doc - 1] : 0;
  // (s and e lie in [0, total_rows] before their difference is looked at)
  const bool bad = s < 0 || e < s || prev > s || e > d.total_rows || (doc == 0 && s != 0) ||
                   (doc == d.n_docs - 1 && e != d.total_rows) || e - s > d.max_seqlen;
  row0 = bad ? 0 : s;
  n = bad ? 0 : e - s;
  return !bad;
}

// For a launch that may begin before the ones that form its records have ended, at the end of its first CTA: a grid
// in which no CTA has waited (every document of one segment) could end before them, and what the stream does next
// would meet them still running.
__device__ __forceinline__ void end_behind_records(const SsmArgs& a) {
  if (a.nseg > 1 && blockIdx.x == 0) tc::grid_dep_wait();
}

// Where the record of segment seg of head h is in the workspace, in records; `start` is the document's first row.
__device__ __forceinline__ long record(const SsmArgs& a, int doc, long start, int seg, int h) {
  return ((a.packed ? start / a.seg_len : static_cast<long>(doc) * (a.nseg - 1)) + seg) * a.H + h;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// The step size of a raw value: softplus(v) = max(v, 0) + log(1 + e^-|v|), which loses nothing at either end.
__device__ __forceinline__ float step_size(float raw, float bias, bool softplus) {
  const float v = raw + bias;
  return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

// 16 bytes of T as floats.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float (&f)[kVec<T>]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&f)[kVec<T>]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(f[i]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace ssm
}  // namespace rapt
