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
// HBM bound: the forward moves 5 tensors, the backward 8, each once. A CTA takes a row at a time (or 8 to
// 32 lanes take a narrow one) and keeps the rows ahead of it in flight in a ring in
// shared memory; each thread copies and reads only its own columns there, so the ring needs no
// barrier. What is missing (columns past the row's end, rows past the last, absent tensors) is zeros
// in the ring, so the arithmetic has no branches. The sums of a row are one reduction: beside r's own
// (sum r^2; backward: also sum t r) it carries sum y^2 of the NEXT row, which that row needs before
// its r, and the backward's sum u yh = sum e g, with e = s a n the joined term, is split by g's terms,
//     sum e g = sum e dr + rho sum e t - rho^2 mean(t rh) sum e r,
// so that it needs no g and no reduction of its own; the rounding of every term stays relative to the
// terms that g itself adds. With ws = w_post s and G = sum_rows a yh g the gain gradients are
// dw_post = s G and ds = w_post G: one column sum serves both. Every thread owns the same columns of
// every row: gains and column sums stay in registers (the sums in fp32, over the CTA's rows). The
// partial sums go to the workspace, one row per CTA, and a second small launch adds them in CTA order:
// no atomics, the same bits every time. Arithmetic is fp32 (two values per instruction where there is
// one); h is formed from the unrounded r and every output is rounded once.
#pragma once

#include <algorithm>
#include <atomic>

#include "activation.cuh"
#include "kernels.h"

namespace rapt {
namespace rn {

// ---------------------------------------------------------------- two fp32 values per instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---------------------------------------------------------------- a thread's columns
// Four values of a thread, as pairs.
struct alignas(16) Quad {
  float2 p[2];
};
__device__ __forceinline__ Quad quad(float x) { return {{both(x), both(x)}}; }
__device__ __forceinline__ Quad operator*(Quad a, Quad b) { return {{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1])}}; }
__device__ __forceinline__ Quad operator*(Quad a, float b) { return a * quad(b); }
__device__ __forceinline__ Quad fma4(Quad a, Quad b, Quad c) {
  return {{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1])}};
}
// s + a . b, the two halves of a pair apart
__device__ __forceinline__ float2 dot4(Quad a, Quad b, float2 s) { return fma2(a.p[1], b.p[1], fma2(a.p[0], b.p[0], s)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// How rows lie: in whole 16-byte vectors, or (D not a multiple of a vector) starting somewhere inside
// one. In the second case all rows of a thread start at the same place in a vector (a launch's rows of a
// thread lie a multiple of a vector's elements apart), `shift` columns into it, and the thread's vectors
// begin that much earlier: the first of a row holds the end of the row before, which is not looked at.
// So every row moves in 16-byte pieces, and only a row's ends are stored otherwise. Forward / backward,
// us, D = 1001, 128 MiB a tensor: bf16 132 / 266, fp32 121 / 197 (copies of a word each: 198 / 334 and
// 153 / 219; D = 1000: 116 / 197 and 118 / 178). Where a row is only part of a warp every warp has ends to
// store: bf16, D = 65: 311 / 497.
enum class Rows { Whole, Shifted };

// Thread tx of a row's tpr owns 4 NC columns, as 16-byte pieces: piece i starts at column
// (i tpr + tx) kPer - shift, so that a warp's accesses are contiguous. RING false: no ring (the rows are
// too wide for one); what would be read there is read from the row itself. Rows are given by the address
// of column 0. FULL: whole rows with D = 4 NC tpr, so that no piece needs a check.
template <typename T, Rows R, int NC, bool RING, bool FULL = false>
struct Cols {
  static constexpr int kBytes = 16;                // of a piece
  static constexpr int kPer = kBytes / sizeof(T);  // columns of a piece
  static constexpr int kPieces = 4 * NC / kPer;
  int tx, tpr, D, shift;
  uint32_t pitch;    // ring bytes of one piece of every thread
  // bf16, few columns a thread: the bits of the first piece that are this row's (elsewhere four more
  // registers cost more than what they save)
  static constexpr bool kMasks = R == Rows::Shifted && sizeof(T) == 2 && NC == 2;
  uint32_t head[4];

  // row0: the first of this thread's rows.
  __device__ __forceinline__ Cols(int tx_, int tpr_, int D_, long row0)
      : tx(tx_), tpr(tpr_), D(D_), shift(R == Rows::Shifted ? static_cast<int>(row0 * D_ & (kPer - 1)) : 0),
        pitch(blockDim.x * kBytes) {
#pragma unroll
    for (int q = 0; q < (kMasks ? 4 : 0); ++q) {
      const int e = col(0) + 2 * q;
      head[q] = e >= 0 ? ~0u : e == -1 ? 0xffff0000u : 0u;
    }
  }
  // Ring bytes of a thread in one stage of `tensors` rows. The threads' places lie side by side, piece
  // by piece: a warp's copies then arrive as whole lines (a thread's places together made the copies
  // 16-byte writes and the fp32 forward a third slower).
  static __host__ __device__ constexpr int stride(int tensors) { return tensors * kPieces * kBytes; }
  __device__ __forceinline__ int col(int i) const { return (i * tpr + tx) * kPer - shift; }
  // Whether piece i lies in the row from end to end.
  __device__ __forceinline__ bool whole(int i) const {
    return R == Rows::Whole || (col(i) >= 0 && col(i) + kPer <= D);
  }
  __device__ __forceinline__ bool has(int e) const {
    return FULL || static_cast<unsigned>(e) < static_cast<unsigned>(D);
  }
  // Place of piece i of tensor slot k, given this thread's first place in a stage.
  __device__ __forceinline__ uint8_t* at(uint8_t* stage, int k, int i) const { return stage + (k * kPieces + i) * pitch; }
  // Zeros in a tensor slot that nothing is copied to.
  __device__ __forceinline__ void clear(uint8_t* stage, int k) const {
    if constexpr (RING) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) *reinterpret_cast<uint4*>(at(stage, k, i)) = make_uint4(0, 0, 0, 0);
    }
  }
  // Starts the copies of this thread's columns of a row into a tensor slot (columns past the end keep the
  // zeros of `clear`).
  __device__ __forceinline__ void fetch(uint8_t* stage, int k, const T* row) const {
#pragma unroll
    for (int i = 0; i < (RING ? kPieces : 0); ++i) {
      const int e = col(i);
      if (!FULL && e >= D) continue;
      const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(at(stage, k, i)));
      if (R == Rows::Whole || e + kPer <= D)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + e) : "memory");
      else  // no further than the row: what follows the last one may be no one's
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(row + e),
                     "r"((D - e) * static_cast<int>(sizeof(T)))
                     : "memory");
    }
  }
  // This thread's columns of a row (null: zeros), from its tensor slot; zeros where there is no column.
  __device__ __forceinline__ void read(uint8_t* stage, int k, const T* row, Quad (&f)[NC]) const {
    float v[4 * NC];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      uint32_t w[4] = {};
      const int e = col(i);
      if constexpr (RING) {
        *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(at(stage, k, i));
        if (R == Rows::Shifted && i == 0) {  // not the end of the row before
          if constexpr (kMasks) {
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] &= head[q];
          } else if (e < 0) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int c = e + q * kPer / 4;
              w[q] = c >= 0 ? w[q] : sizeof(T) == 2 && c == -1 ? w[q] & 0xffff0000u : 0u;
            }
          }
        }
      } else if (row != nullptr && e < D) {
        if (whole(i)) {
          *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(row + e);
        } else {
#pragma unroll
          for (int q = 0; q < kPer; ++q)
            if (has(e + q)) {
              if constexpr (sizeof(T) == 4)
                w[q] = reinterpret_cast<const uint32_t*>(row)[e + q];
              else
                w[q / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[e + q]) << (16 * (q % 2));
            }
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 4) {
          v[i * kPer + q] = __uint_as_float(w[q]);
        } else {
          v[i * kPer + 2 * q] = __uint_as_float(w[q] << 16);
          v[i * kPer + 2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
      f[c] = {{make_float2(v[4 * c], v[4 * c + 1]), make_float2(v[4 * c + 2], v[4 * c + 3])}};
  }
  // Stores this thread's columns to a row (none where it is null).
  __device__ __forceinline__ void write(T* row, const Quad (&f)[NC]) const {
    if (row == nullptr) return;
    float v[4 * NC];
    flat(f, v);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int e = col(i);
      if (!FULL && e >= D) continue;
      const float* q = v + i * kPer;
      if constexpr (sizeof(T) == 4) {
        if (whole(i)) {
          *reinterpret_cast<float4*>(row + e) = make_float4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (has(e + k)) row[e + k] = q[k];
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pack_bf16(q[2 * k], q[2 * k + 1]);
        if (whole(i)) {
          *reinterpret_cast<uint4*>(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {  // words, but for a first or last column that shares one with another row
          const int first = max(0, (1 - e) / 2), words = (D - e) / 2 - first;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (static_cast<unsigned>(k - first) < static_cast<unsigned>(max(words, 0)))
              *reinterpret_cast<uint32_t*>(row + e + 2 * k) = w[k];
          uint16_t* const h = reinterpret_cast<uint16_t*>(row);
          const auto word = [&](int k) { return k < 2 ? (k == 0 ? w[0] : w[1]) : k == 2 ? w[2] : w[3]; };
          if (e < 0 && (e & 1)) h[0] = static_cast<uint16_t>(word(-e / 2) >> 16);
          if (e + kPer > D && ((D - e) & 1)) h[D - 1] = static_cast<uint16_t>(word((D - e) / 2));
        }
      }
    }
  }
  static __device__ __forceinline__ void flat(const Quad (&f)[NC], float (&v)[4 * NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      v[4 * c] = f[c].p[0].x;
      v[4 * c + 1] = f[c].p[0].y;
      v[4 * c + 2] = f[c].p[1].x;
      v[4 * c + 3] = f[c].p[1].y;
    }
  }
  // The gains of this thread's columns: ones where there is no gain or no column.
  __device__ __forceinline__ void gain(const float* w, Quad (&f)[NC]) const {
    float v[4 * NC];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int e = col(i) + k;
        v[i * kPer + k] = w != nullptr && has(e) ? w[e] : 1.f;
      }
#pragma unroll
    for (int c = 0; c < NC; ++c)
      f[c] = {{make_float2(v[4 * c], v[4 * c + 1]), make_float2(v[4 * c + 2], v[4 * c + 3])}};
  }
  // fp32 column sums to a row of partials.
  __device__ __forceinline__ void put_sums(float* row, const Quad (&f)[NC]) const {
    float v[4 * NC];
    flat(f, v);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (has(col(i) + k)) row[col(i) + k] = v[i * kPer + k];
  }
};

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have arrived (N < 0: there are none).
template <int N>
__device__ __forceinline__ void wait_copies() {
  if constexpr (N >= 0) asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- reductions
// Sums eight values over a warp: lane 4 v ends with the sum of value v. Halving the values with the
// distance takes 9 shuffles where one value at a time takes 40.
__device__ __forceinline__ float warp_sum8(const float (&v)[8]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool up = lane & 16;
    a[i] = (up ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 4], 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool up = lane & 8;
    b[i] = (up ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, up ? a[i] : a[i + 2], 8);
  }
  const bool up = lane & 4;
  c = (up ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, up ? b[0] : b[1], 4);
  c += __shfl_xor_sync(0xffffffffu, c, 2);
  return c + __shfl_xor_sync(0xffffffffu, c, 1);
}

// Sums N <= 6 values over the threads of a row. A row of 8, 16 or 32 lanes uses shuffles alone; a row of
// a whole CTA adds the warps' sums from `red` (two alternating halves, so one barrier per call
// suffices: a half is rewritten two calls later, after a barrier that follows its last read).
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int tpr, float (*red)[32][8], int& half) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5;
  if (tpr < 32) {
    for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    return;
  }
  if constexpr (N <= 2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[half][warp][n] = v[n];
    }
  } else {
    float w[8] = {};
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = v[n];
    const float c = warp_sum8(w);
    if (warps == 1) {
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, c, 4 * n);
      return;
    }
    if ((lane & 3) == 0) red[half][warp][lane >> 2] = c;
  }
  __syncthreads();
  // lane 8 j + n adds value n of the warps j, j + 4, ...
  float c = 0.f;
  for (int j = lane >> 3; j < warps; j += 4) c += red[half][j][lane & 7];
  c += __shfl_xor_sync(0xffffffffu, c, 8);
  c += __shfl_xor_sync(0xffffffffu, c, 16);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, c, n);
  half ^= 1;
}

// x^(-1/2) within 2^-22.
__device__ __forceinline__ float inv_root(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// act(z) (ones without a gate) and act'(z) over a thread's columns.
template <bool GRAD, int NC>
__device__ __forceinline__ void act_cols(bool gated, Act act, const Quad (&z)[NC], Quad (&a)[NC], Quad (&da)[NC]) {
  if (!gated) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      a[c] = quad(1.f);
      if (GRAD) da[c] = quad(0.f);
    }
    return;
  }
  if (act == Act::Sigmoid || act == Act::Silu) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x = z[c].p[i];
        float2 s, e;
        s.x = GRAD ? sigmoid_f(x.x, e.x) : sigmoid_f(x.x);
        s.y = GRAD ? sigmoid_f(x.y, e.y) : sigmoid_f(x.y);
        const float2 t = GRAD ? mul2(e, s) : s;  // 1 - s
        if (act == Act::Sigmoid) {
          a[c].p[i] = s;
          if (GRAD) da[c].p[i] = mul2(s, t);
        } else {
          a[c].p[i] = mul2(x, s);
          if (GRAD) da[c].p[i] = mul2(s, fma2(x, t, both(1.f)));
        }
      }
    return;
  }
  if (act == Act::Gelu) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 p, d;
        gelu_two<GRAD>(z[c].p[i], p, d);
        a[c].p[i] = p;
        if (GRAD) da[c].p[i] = d;
      }
    return;
  }
  float zz[4 * NC], aa[4 * NC], dd[4 * NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    zz[4 * c] = z[c].p[0].x;
    zz[4 * c + 1] = z[c].p[0].y;
    zz[4 * c + 2] = z[c].p[1].x;
    zz[4 * c + 3] = z[c].p[1].y;
  }
  if (act == Act::Relu) {
#pragma unroll
    for (int i = 0; i < 4 * NC; ++i) act_one<GRAD>(Act::Relu, zz[i], aa[i], dd[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * NC; ++i) act_one<GRAD>(Act::None, zz[i], aa[i], dd[i]);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    a[c] = {{make_float2(aa[4 * c], aa[4 * c + 1]), make_float2(aa[4 * c + 2], aa[4 * c + 3])}};
    if (GRAD) da[c] = {{make_float2(dd[4 * c], dd[4 * c + 1]), make_float2(dd[4 * c + 2], dd[4 * c + 3])}};
  }
}

// w_post s and w_pre of a thread's columns.
template <int NC, typename C>
__device__ __forceinline__ void load_gains(const ResidualNormArgs& a, const C& in, Quad (&ws)[NC], Quad (&wpre)[NC]) {
  in.gain(a.w_post, ws);
  in.gain(a.scale, wpre);
#pragma unroll
  for (int c = 0; c < NC; ++c) ws[c] = ws[c] * wpre[c];
  in.gain(a.w_pre, wpre);
}

constexpr int kFwdTensors = 3, kBwdTensors = 5;

// Threads of a row (tpr: 8, 16 or 32 lanes of a warp, or a CTA of whole warps) and of a CTA, for ept
// columns a thread, where a row takes up to `more` columns of another one with it.
struct RowShape {
  int ept, tpr, threads;
};
inline RowShape row_shape(int D, int ept, int more) {
  const int need = (D + more + ept - 1) / ept;
  RowShape s;
  s.ept = ept;
  s.tpr = need <= 8 ? 8 : need <= 16 ? 16 : (need + 31) / 32 * 32;
  s.threads = s.tpr > 32 ? s.tpr : ept == 8 ? 256 : 128;
  return s;
}
// Columns a thread of the backward: as many as keep a CTA at 512 threads, for their registers (D = 5120
// in fp32: 242 us with eight, 204 with sixteen); the widest rows that are no whole vectors take 704 of
// twenty-four (bf16, D = 16383: 1050 us, 1150 with thirty-two). bf16 takes sixteen from 257 to 2048, too, where that
// leaves few lanes idle or a row to a warp: fewer instructions a value (D = 2048: 197 -> 186 us).
inline RowShape bwd_shape(int D, int more, bool f32) {
  const int n = D + more;
  const RowShape s16 = row_shape(D, 16, more);
  if (n <= 4096) {
    const bool fits = n > 256 && n <= 2048 && (s16.tpr == 32 || (more == 0 && s16.tpr * 16 * 7 <= n * 8));
    return !f32 && fits ? s16 : row_shape(D, 8, more);
  }
  return n <= 8192 ? s16 : row_shape(D, n <= 12288 || more > 0 ? 24 : 32, more);
}
// CTAs of a backward launch at most (its registers hold an SM to 1024 threads): the workspace's rows
// of partial sums.
inline int max_parts(const RowShape& s) { return 160 * std::max(1, 1024 / s.threads); }

constexpr size_t kSmemMost = 224 * 1024;  // shared memory that a CTA may ask for beside its 2 KB of sums

// Bytes of a ring of `stages` rows of `tensors` tensors.
template <typename T, Rows R, int NC>
size_t ring_bytes(const RowShape& s, int stages, int tensors) {
  return static_cast<size_t>(stages) * Cols<T, R, NC, true>::stride(tensors) * s.threads;
}

// `apart`: what the number of rows between a thread's rows is to be a multiple of.
template <auto KERNEL, typename ARGS>
cudaError_t launch_rows(const ARGS& a, const RowShape& s, size_t smem, int most, int apart, int* grid,
                        cudaStream_t stream) {
  const long slots = s.threads / s.tpr, ctas = (a.T + slots - 1) / slots;
  int per_sm = 1, sms = 0, dev = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  static std::atomic<unsigned long long> configured{0};  // bit per device
  if (e == cudaSuccess && (dev >= 64 || !((configured.load(std::memory_order_relaxed) >> dev) & 1ull))) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemMost));
    if (e == cudaSuccess && dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  // all CTAs are resident at once: the rows ahead are then the whole GPU's
  if (e == cudaSuccess && ctas > sms)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, s.threads, smem);
  if (e != cudaSuccess) return e;
  *grid = static_cast<int>(std::min<long>({ctas, static_cast<long>(sms) * std::max(1, per_sm), most}));
  const int unit = static_cast<int>(std::max<long>(apart / slots, 1));  // both powers of two
  if (*grid < ctas) *grid = static_cast<int>(std::min<long>(ctas, std::max(*grid / unit, 1) * unit));
  KERNEL<<<*grid, s.threads, smem, stream>>>(a, s.tpr);
  note_launches(1);
  return cudaGetLastError();
}

// How the rows of a [T, D] tensor lie, and the columns that one may take with it.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));
template <typename T>
bool whole_rows(int D) {
  return D % kVec<T> == 0;
}
template <typename T, Rows R>
constexpr int kMore = R == Rows::Shifted ? kVec<T> - 1 : 0;

}  // namespace rn
}  // namespace rapt
