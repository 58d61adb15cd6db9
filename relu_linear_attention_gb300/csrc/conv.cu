// The short causal convolution of every channel over its document's tokens, with its activation (sm_103a):
//   y[t, c] = act(b[c] + sum_{k<W} w[c, k] x[t - W + 1 + k, c]),  W <= 4.
//
// HBM bound: every token is read and written once. A thread owns V = 4 channels (8 bytes in bf16; with 16 the taps,
// the window and the values in flight took 184 registers and 141 us for 16384 x 4352, 64 so) and walks up to 64 tokens
// with the last W - 1 of them in registers; kAhead loads fly while the kAhead tokens before them are computed (54 us
// of that case, 79 % of a copy; 30011 packed tokens x 1537 fp32: 72 us). The W - 1 tokens before its first come from
// L2, where the tile before has put them. Where a tile ends follows from how many tiles fill the GPU. A document's
// tokens in the tile are one run without checks; at its first token the window is its carried state. Rows of no whole
// 4 channels go channel by channel. The last W - 1 inputs of each document are written by threads behind the tiles of
// the same launch.
#include "ssm.cuh"

namespace rapt {
namespace {

using namespace ssm;

constexpr int kThreads = 128;
constexpr int kAhead = 8;
enum Path { kNone, kSilu, kAny };  // of the activation: the usual ones have no choice in the loop

// Values in flight: V = 1, or 4 channels.
template <typename T, int V>
struct Raw {
  uint32_t w[sizeof(T) * V <= 4 ? 1 : sizeof(T) * V / 4];
};
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> fetch(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 1 && sizeof(T) == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (V == 1) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (sizeof(T) == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void widen_raw(const Raw<T, V>& r, float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (sizeof(T) == 4) f[v] = __uint_as_float(r.w[v]);
    else f[v] = __uint_as_float(v % 2 == 0 ? r.w[v / 2] << 16 : r.w[v / 2] & 0xffff0000u);
  }
}
template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&f)[V]) {
  widen_raw<T, V>(fetch<T, V>(p), f);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&f)[V]) {
  if constexpr (V == 1) *p = from_float<T>(f[0]);
  else store4(p, f[0], f[1], f[2], f[3]);
}

// The taps of a thread's channels, [V, W] side by side in w.
template <int V, int W>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int c, float (&taps)[W][V], float (&b)[V]) {
  float f[V * W];
  const float* p = w + static_cast<long>(c) * W;
#pragma unroll
  for (int i = 0; i < V * W; i += V == 1 ? 1 : 4) {
    if constexpr (V == 1) {
      f[i] = p[i];
    } else {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      f[i] = q.x, f[i + 1] = q.y, f[i + 2] = q.z, f[i + 3] = q.w;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) taps[k][v] = f[v * W + k];
    b[v] = bias != nullptr ? bias[c + v] : 0.f;
  }
}
template <int V, Path PATH>
__device__ __forceinline__ void activate(Act act, float (&y)[V]) {
  if constexpr (PATH == kSilu) {
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] *= sigmoid_f(y[v]);
  } else if constexpr (PATH == kAny) {
    float unused;
#pragma unroll
    for (int v = 0; v < V; ++v) act_one<false>(act, y[v], y[v], unused);
  }
}

// The document of row t: the last one that begins at t or before.
__device__ __forceinline__ int find_doc(const Docs& d, int t) {
  if (d.cu_seqlens == nullptr) return t / d.doc_len;
  int lo = 0, hi = d.n_docs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (d.cu_seqlens[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ void bounds(const Docs& d, int doc, int& start, int& end) {
  if (d.cu_seqlens == nullptr) {
    start = doc * d.doc_len;
    end = start + d.doc_len;
  } else {
    start = max(d.cu_seqlens[doc], 0);
    end = min(d.cu_seqlens[doc + 1], d.total_rows);
  }
}

// The last W - 1 inputs of a document; without state_final, a document an item, a look at its bounds alone.
template <typename T, int V, int W>
__device__ __forceinline__ void last_inputs(const ConvArgs& a, long i, int nvec) {
  const int per_doc = a.state_final != nullptr ? nvec : 1;
  const int doc = static_cast<int>(i / per_doc), c = static_cast<int>(i % per_doc) * V;
  long row0;
  int n;
  const bool good = doc_rows(a.docs, doc, row0, n);
  if (!good && c == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, 1u);
  if (!good || a.state_final == nullptr) return;
  const T* x = static_cast<const T*>(a.x);
  const T* old = static_cast<const T*>(a.state);
  T* dst = static_cast<T*>(a.state_final);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = n - (W - 1) + k;  // may be before the document
    float f[V] = {};
    if (t >= 0) load<T, V>(x + (row0 + t) * a.x_stride + c, f);
    else if (old != nullptr) load<T, V>(old + (static_cast<long>(doc) * (W - 1) + (t + W - 1)) * a.D + c, f);
    store<T, V>(dst + (static_cast<long>(doc) * (W - 1) + k) * a.D + c, f);
  }
}

template <typename T, int V, int W, Path PATH>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvArgs a, int nvec, int tokens, long tiles, long items) {
  const long item = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
  if (item >= items) return;
  if (item >= tiles) {
    last_inputs<T, V, W>(a, item - tiles, nvec);
    return;
  }
  const int c = static_cast<int>(item % nvec) * V;
  const int t0 = static_cast<int>(item / nvec) * tokens, t1 = min(t0 + tokens, a.docs.total_rows);
  const T* const x0 = static_cast<const T*>(a.x) + c;
  float w[W][V], b[V];
  load_taps<V, W>(a.w, a.bias, c, w, b);
  int doc = find_doc(a.docs, t0), start, end;
  bounds(a.docs, doc, start, end);
  float win[W - 1][V];  // the W - 1 inputs before token t of the document at hand
  const auto carried = [&](int k, float (&f)[V]) {  // row k of the document's state
#pragma unroll
    for (int v = 0; v < V; ++v) f[v] = 0.f;
    if (a.state != nullptr)
      load<T, V>(static_cast<const T*>(a.state) + (static_cast<long>(doc) * (W - 1) + k) * a.D + c, f);
  };
#pragma unroll
  for (int k = 0; k < W - 1; ++k) {
    const int t = t0 - (W - 1) + k;
    if (t >= start && t >= 0) load<T, V>(x0 + t * a.x_stride, win[k]);
    else carried(min(max(t - start + W - 1, 0), W - 2), win[k]);
  }
  const auto one = [&](const Raw<T, V>& raw, T* to) {
    float cur[V], y[V];
    widen_raw<T, V>(raw, cur);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      y[v] = b[v];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) y[v] = fmaf(w[k][v], win[k][v], y[v]);
      y[v] = fmaf(w[W - 1][v], cur[v], y[v]);
    }
    activate<V, PATH>(a.act, y);
    store<T, V>(to, y);
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k + 1 < W - 1; ++k) win[k][v] = win[k + 1][v];
      win[W - 2][v] = cur[v];
    }
  };
  int t = t0;
  while (t < t1) {
    if (t >= end) {  // the next document that has this token
      while (t >= end && doc + 1 < a.docs.n_docs) {
        ++doc;
        bounds(a.docs, doc, start, end);
      }
      if (t >= end) break;  // (there is none in a malformed cu_seqlens)
#pragma unroll
      for (int k = 0; k < W - 1; ++k) carried(k, win[k]);
    }
    if (t < start) {
      t = start;
      continue;
    }
    int n = min(t1, end) - t;
    const T* x = x0 + t * a.x_stride;
    T* out = static_cast<T*>(a.out) + static_cast<long>(t) * a.D + c;
    t += n;
    if (n >= kAhead) {
      Raw<T, V> raw[kAhead], next[kAhead];
      const auto load_ahead = [&](Raw<T, V>(&to)[kAhead]) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          to[j] = fetch<T, V>(x);
          x += a.x_stride;
        }
      };
      load_ahead(raw);
      for (bool more = true; more; n -= kAhead) {
        more = n >= 2 * kAhead;
        if (more) load_ahead(next);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          one(raw[j], out);
          out += a.D;
          raw[j] = next[j];
        }
      }
    }
#pragma unroll 1
    for (; n > 0; --n) {
      one(fetch<T, V>(x), out);
      x += a.x_stride;
      out += a.D;
    }
  }
}

// One token: the window is the state's rows, shifted by the new token.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const T* x, long x_stride, const float* w, const float* bias, T* state, T* out, int N, int D,
                     Act act, int nvec) {
  const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= static_cast<long>(N) * nvec) return;
  const int n = static_cast<int>(i / nvec), c = static_cast<int>(i % nvec) * V;
  float win[W][V], taps[W][V], y[V];
  load_taps<V, W>(w, bias, c, taps, y);
  T* s = state + static_cast<long>(n) * (W - 1) * D + c;
#pragma unroll
  for (int k = 0; k < W - 1; ++k) load<T, V>(s + static_cast<long>(k) * D, win[k]);
  load<T, V>(x + n * x_stride + c, win[W - 1]);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < W; ++k) y[v] = fmaf(taps[k][v], win[k][v], y[v]);
  activate<V, kAny>(act, y);
  store<T, V>(out + static_cast<long>(n) * D + c, y);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) store<T, V>(s + static_cast<long>(k) * D, win[k + 1]);
}

template <typename T, int V, int W, Path PATH>
cudaError_t go(const ConvArgs& a, cudaStream_t stream) {
  const int nvec = a.D / V;
  // tokens a thread: as many as leave the GPU 1024 threads an SM
  int tokens = 64;
  const auto count = [&] { return (static_cast<long>(a.docs.total_rows) + tokens - 1) / tokens * nvec; };
  while (tokens > kAhead && count() < 152L * 1024) tokens /= 2;
  const long tiles = count();
  // (documents are looked through for a malformed cu_seqlens, too)
  const bool look = a.docs.cu_seqlens != nullptr && a.docs.dev_status != nullptr;
  const long items = tiles + static_cast<long>(a.docs.n_docs) * (a.state_final != nullptr ? nvec : look ? 1 : 0);
  if (items == 0) return cudaSuccess;
  const long grid = (items + kThreads - 1) / kThreads;
  conv_kernel<T, V, W, PATH><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a, nvec, tokens, tiles, items);
  note_launches(1);
  return cudaGetLastError();
}
template <typename T, int V, int W>
cudaError_t by_act(const ConvArgs& a, cudaStream_t s) {
  return a.act == Act::Silu   ? go<T, V, W, kSilu>(a, s)
         : a.act == Act::None ? go<T, V, W, kNone>(a, s)
                              : go<T, V, W, kAny>(a, s);
}
template <typename T, int V, int W>
cudaError_t go_step(const void* x, long xs, const float* w, const float* bias, void* state, void* out, int N, int D,
                    Act act, cudaStream_t stream) {
  const int nvec = D / V;
  const long grid = (static_cast<long>(N) * nvec + kThreads - 1) / kThreads;
  conv_step_kernel<T, V, W><<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(
      static_cast<const T*>(x), xs, w, bias, static_cast<T*>(state), static_cast<T*>(out), N, D, act, nvec);
  note_launches(1);
  return cudaGetLastError();
}
// Whole pieces of 4 channels: every row and every token of a state begins at a multiple of them.
bool whole(int D, long stride) { return D % 4 == 0 && stride % 4 == 0; }
template <typename T>
cudaError_t pick(const ConvArgs& a, cudaStream_t s) {
  if (whole(a.D, a.x_stride))
    return a.W == 2 ? by_act<T, 4, 2>(a, s) : a.W == 3 ? by_act<T, 4, 3>(a, s) : by_act<T, 4, 4>(a, s);
  return a.W == 2 ? by_act<T, 1, 2>(a, s) : a.W == 3 ? by_act<T, 1, 3>(a, s) : by_act<T, 1, 4>(a, s);
}
template <typename T>
cudaError_t pick_step(const void* x, long xs, const float* w, const float* bias, void* st, void* out, int N, int D,
                      int W, Act act, cudaStream_t s) {
  constexpr int V = 4;
  if (whole(D, xs))
    return W == 2   ? go_step<T, V, 2>(x, xs, w, bias, st, out, N, D, act, s)
           : W == 3 ? go_step<T, V, 3>(x, xs, w, bias, st, out, N, D, act, s)
                    : go_step<T, V, 4>(x, xs, w, bias, st, out, N, D, act, s);
  return W == 2   ? go_step<T, 1, 2>(x, xs, w, bias, st, out, N, D, act, s)
         : W == 3 ? go_step<T, 1, 3>(x, xs, w, bias, st, out, N, D, act, s)
                  : go_step<T, 1, 4>(x, xs, w, bias, st, out, N, D, act, s);
}

}  // namespace

cudaError_t launch_conv(DType dt, const ConvArgs& a, cudaStream_t stream) {
  return dt == DType::F32 ? pick<float>(a, stream) : pick<__nv_bfloat16>(a, stream);
}
cudaError_t launch_conv_step(DType dt, const void* x, long x_stride, const float* w, const float* bias, void* state,
                             void* out, int N, int D, int W, Act act, cudaStream_t stream) {
  return dt == DType::F32 ? pick_step<float>(x, x_stride, w, bias, state, out, N, D, W, act, stream)
                          : pick_step<__nv_bfloat16>(x, x_stride, w, bias, state, out, N, D, W, act, stream);
}

}  // namespace rapt
