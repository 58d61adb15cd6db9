// The selective scan in chunks on the 5th-generation tensor cores (tcgen05 + TMEM), sm_103a: bf16, P and N of 64 or
// 128, fp32 accumulation, decays and states.
//
//   S_t = e^(a_t) S_{t-1} + dt_t B_t x_t^T,  a_t = dt_t A <= 0,  y_t = (S_t^T C_t + D x_t) silu(z_t)
//
// A CTA walks the 128-token chunks of a segment of a document with two heads of 64 columns (or one of 128) that
// share B and C. With s_i = a_1 + ... + a_i inside the chunk and h the state before it, and sg_i = max(e^(s_i), 2^-64):
//
//   G  = C B^T                              (128 x 128)  once for both heads
//   M  = G_ij e^(s_i - s_j) dt_j / sg_i     (j <= i; rounded to bf16, written over G in TMEM)
//   Y  = C h^T + M x,  y_i = sg_i Y_i       (128 x 128)  one accumulator; h a bf16 copy of the state, [columns, N]
//   h <- e^(s_128) h + xw^T B               (128 x N)    xw_j = e^(s_128 - s_j) dt_j x_j in two bf16 parts, in TMEM
//
// Taking sg_i out of both products lets them share an accumulator: where a row's decay is below 2^-64, C h counts
// 2^-64 for 0. Two bf16 parts of xw (16 bits) keep the fp32 state to 2^-17 of its terms: with one part it would be
// 2^-9, and the state is an output and the start of everything later. B and x enter exactly as they are.
//
// Decays are formed from sums inside blocks of 32 tokens, so that a difference of logarithms is that of sums of at
// most 32 and what lies between: left of the diagonal block, e^(s_i - s_j) = e^(s_i - s at the end of j's block) x
// e^(that - s_j), one factor a row and block and one a column, both at most 1: no exponential an element, no
// overflow at any decay. On the diagonal block each element has its own. a_t stops at -160 log 2 (2^-160 is 0).
//
// Warps (640 threads, one CTA an SM):
//   0-7   rows:   G -> M (a TMEM lane quarter and every other block of 32 keys each), then the epilogue of half of
//                 the tile's columns: y in the place of x in shared memory, from where the TMA stores it;
//   8-15  states: the increment into h (fp32, in registers) and its bf16 copy in shared memory, then xw of half of the
//                 next chunk's tokens (a lane is a column of x);
//   16    MMA issue, 17 TMA loads and stores, 18-19 step sizes, decays and their sums, one head each.
// Shared memory: two x and two B tiles, one C tile, the state copy, the decay tables. A document is cut into
// segments where there are fewer units than SMs; kernel A (the same code without reading) gives their increments.
// Every wait is bounded; one that gives up sets RAPT_DEV_INTERNAL and the CTA winds down.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "ssm.cuh"
#include "tc_features.cuh"
#include "tc_utils.cuh"
#include "tensor_map.h"

namespace rapt {
namespace {

using namespace ssm;

constexpr int kC = 128;                       // tokens of a chunk
constexpr int kRows = 256, kStates = 256;     // threads of the two groups
constexpr int kThreads = kRows + kStates + 128;
constexpr int kWarpIssue = (kRows + kStates) / 32, kWarpTma = kWarpIssue + 1, kWarpTab = kWarpIssue + 2;
constexpr long long kWaitCycles = 2000000000LL;  // ~1 s
constexpr uint32_t kDevInternal = 2u;
constexpr int kLaunchRegs = 96, kRegsRows = 104, kRegsStates = 112, kRegsRest = 48;
static_assert(kRows * kRegsRows + kStates * kRegsStates + 128 * kRegsRest <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeastLog = -160.f;  // of a token's decay, base 2
constexpr float kLeastRow = -64.f;   // of a row's common factor

// Byte offsets from a 1024-byte aligned base, and TMEM columns.
template <int N>
struct Lay {
  static constexpr uint32_t XT = 32768, NT = N / 64 * 16384;
  static constexpr uint32_t X = 0, B = 2 * XT, C = B + 2 * NT, H = C + NT;
  static constexpr uint32_t TAB = H + NT;  // [2 buffers][p, q, f][2 heads][kC] fp32
  static constexpr uint32_t TAB1 = 3 * 2 * kC * 4;
  static constexpr uint32_t BAR = TAB + 2 * TAB1;
  static constexpr int NBAR = 24;
  static constexpr uint32_t MISC = BAR + NBAR * 8;
  static constexpr uint32_t BYTES = MISC + 16;
  static_assert(BYTES <= 232448, "shared memory budget");
  static constexpr uint32_t TG = 0, TX = 128, TI = 256, TY = 384;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 lds_v4(const uint8_t* sm, uint32_t off) { return *reinterpret_cast<const uint4*>(sm + off); }

// Sum of the block sums b[from .. to).
__device__ __forceinline__ float between(const float (&b)[4], int from, int to) {
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) v += k >= from && k < to ? b[k] : 0.f;
  return v;
}

struct Maps {
  CUtensorMap x, b, c, out;
};

template <int P, int N, bool READ>
__global__ void __launch_bounds__(kThreads, 1) ssm_tc_kernel(const SsmArgs a, const __grid_constant__ Maps maps) {
  using L = Lay<N>;
  constexpr int NH = P == 64 ? 2 : 1;  // heads of a CTA
  constexpr long kRec = static_cast<long>(N) * P + kSsmRecTail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (!READ) tc::grid_launch_dependents();  // the scan may start; it waits for this grid before it reads ws

  const int R = a.H / a.G, per_group = (R + NH - 1) / NH, units = a.G * per_group;
  const int nseg = READ ? a.nseg : a.nseg - 1;
  const int seg = static_cast<int>(blockIdx.x % nseg);
  const int unit = static_cast<int>(blockIdx.x / nseg % units);
  const int at_doc = static_cast<int>(blockIdx.x / nseg / units);
  const int doc = a.order != nullptr ? a.order[at_doc] : at_doc;
  const int g = unit / per_group, h0 = g * R + unit % per_group * NH;
  const int nh = min(NH, g * R + R - h0);  // an odd head of a group is alone
  long row0;
  int n;
  const bool good = doc_rows(a.docs, doc, row0, n);
  if (READ && !good && seg == 0 && unit == 0 && tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, 1u);
  const int segs = n > 0 ? (n + a.seg_len - 1) / a.seg_len : 1;
  if (!good || seg >= (READ ? segs : segs - 1)) return;  // uniform across the CTA, before any allocation
  const int seg_start = seg * a.seg_len, seg_n = min(a.seg_len, n - seg_start);  // 0: an empty document
  const int nchunks = (seg_n + kC - 1) / kC;
  row0 += seg_start;

  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  if (base & 1023u) {  // the swizzled layouts need 1024-byte alignment
    if (tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, kDevInternal);
    return;
  }
  const uint32_t bars = base + L::BAR;
  const uint32_t b_full = bars, x_full = bars + 16, c_full = bars + 32, tab_full = bars + 40, tab_free = bars + 56;
  const uint32_t g_done = bars + 72, m_ready = bars + 80, h_ready = bars + 88, xw_ready = bars + 96;
  const uint32_t inc_done = bars + 104, yoff_done = bars + 112, y_done = bars + 120, y_free = bars + 128;
  const uint32_t staged = bars + 136, drain = bars + 152;
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(smem + L::MISC);
  volatile int* const s_abort = reinterpret_cast<volatile int*>(smem + L::MISC + 4);

  if (warp == 0) {
    tc::tmem_alloc(tc::smem_u32(s_tmem), 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(b_full + 8 * i, 1);
      tc::mbar_init(x_full + 8 * i, 1);
      tc::mbar_init(tab_full + 8 * i, 32 * NH);
      tc::mbar_init(tab_free + 8 * i, READ ? kRows + kStates : kStates);
      tc::mbar_init(staged + 8 * i, kRows);
    }
    tc::mbar_init(c_full, 1);
    tc::mbar_init(g_done, 1);
    tc::mbar_init(m_ready, kRows);
    tc::mbar_init(h_ready, kStates);
    tc::mbar_init(xw_ready, kStates);
    tc::mbar_init(inc_done, 1);
    tc::mbar_init(yoff_done, 1);
    tc::mbar_init(y_done, 1);
    tc::mbar_init(y_free, kRows);
    tc::mbar_init(drain, 1);
    tc::mbar_fence_init();
    *s_abort = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const auto wait = [&](uint32_t bar, int parity) { return tc::mbar_wait(bar, parity, kWaitCycles) && *s_abort == 0; };
  const auto table = [&](int c, int which, int head) {
    return reinterpret_cast<const float*>(smem + L::TAB + (c & 1) * L::TAB1) + (which * 2 + head) * kC;
  };
  const int q4 = warp & 3;  // TMEM lane quarter
  const uint32_t tl = static_cast<uint32_t>(32 * q4) << 16;

  if (warp < kRows / 32) {
    // ============================================================ rows
    tc::regs_inc<kRegsRows>();
    if constexpr (READ) {
      const int hf = warp >> 2;  // keys: the blocks of 32 with this parity; epilogue: this half of the columns
      const int i = 32 * q4 + lane;
      const int eh = NH == 2 ? hf : 0;               // the head of those columns
      const bool live = NH == 1 || hf < nh;
      const int head = h0 + min(eh, nh - 1);
      const float skip = a.D != nullptr ? a.D[head] : 0.f;
      const long ecol = static_cast<long>(head) * P + (NH == 1 ? 64 * hf : 0);
      const __nv_bfloat16* const zg =
          a.z != nullptr ? static_cast<const __nv_bfloat16*>(a.z) + (row0 + i) * a.zs + ecol : nullptr;
      __nv_bfloat16* const og =
          static_cast<__nv_bfloat16*>(a.out) + (row0 + i) * (static_cast<long>(a.H) * P) + ecol;
      int ok = 1;
      for (int c = 0; c < nchunks; ++c) {
        const int s = c & 1, ph = (c >> 1) & 1;
        ok = wait(tab_full + 8 * s, ph);
        // this row's sums: pl = p_i - log2 sg_i; bs = the block sums
        float pl[NH], bs[NH][4], sg = 0.f;
#pragma unroll
        for (int k = 0; k < NH; ++k) {
          const float* const p = table(c, 0, k);
#pragma unroll
          for (int J = 0; J < 4; ++J) bs[k][J] = p[32 * J + 31];
          const float own = p[i], ls = fmaxf(own + between(bs[k], 0, q4), kLeastRow);
          pl[k] = own - ls;
          if (k == eh) sg = ex2(ls);
        }
        ok = ok && wait(g_done, c & 1);
        if (__any_sync(0xffffffffu, !ok)) break;  // warp-uniform: TMEM accesses stay converged
        tc::fence_after_sync();
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int J = hf + 2 * jj;
          const uint32_t tg = tmem + tl + L::TG + 32 * J;
          if (J > q4) {
            uint32_t zero[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) zero[e] = 0u;
            tc::tmem_st16(tg, zero);
            if (NH == 2) tc::tmem_st16(tg + 16, zero);
            continue;
          }
          uint32_t u[2][16];
          tc::tmem_ld16(tg, u[0]);
          tc::tmem_ld16(tg + 16, u[1]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < NH; ++k) {
            uint32_t w[16];
            if (J == q4) {
              const float* const q = table(c, 1, k) + 32 * J;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(q + e);
                const float qq[4] = {v.x, v.y, v.z, v.w};
                float m[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                  const float x = __uint_as_float(u[e / 16][e % 16 + d]) * ex2(pl[k] - qq[d]);
                  m[d] = e + d <= lane ? x : 0.f;
                }
                w[e / 2] = tc::pack_bf16x2(m[0], m[1]);
                w[e / 2 + 1] = tc::pack_bf16x2(m[2], m[3]);
              }
            } else {
              const float* const f = table(c, 2, k) + 32 * J;
              const float rf = ex2(pl[k] + between(bs[k], J + 1, q4));
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = *reinterpret_cast<const float4*>(f + e);
                const float2 r2 = make_float2(rf, rf);
                const float2 m0 = __fmul2_rn(
                    __fmul2_rn(make_float2(__uint_as_float(u[e / 16][e % 16]), __uint_as_float(u[e / 16][e % 16 + 1])), r2),
                    make_float2(v.x, v.y));
                const float2 m1 = __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(u[e / 16][e % 16 + 2]),
                                                                    __uint_as_float(u[e / 16][e % 16 + 3])), r2),
                                             make_float2(v.z, v.w));
                w[e / 2] = tc::pack_bf16x2(m0.x, m0.y);
                w[e / 2 + 1] = tc::pack_bf16x2(m1.x, m1.y);
              }
            }
            tc::tmem_st16(tg + 16 * k, w);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(m_ready);
        tc::mbar_arrive(tab_free + 8 * s);
        // the epilogue of this row's 64 columns
        const int lt = c * kC + i;
        uint4 z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          z[e] = zg != nullptr && live && lt < seg_n
                     ? __ldg(reinterpret_cast<const uint4*>(zg + static_cast<long>(c) * kC * a.zs) + e)
                     : make_uint4(0, 0, 0, 0);
        const bool whole = c * kC + kC <= seg_n;
        const uint32_t xo = L::X + s * L::XT + hf * 16384;
        ok = wait(x_full + 8 * s, ph) && wait(y_done, c & 1);
        if (__any_sync(0xffffffffu, !ok)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t u[2][16];
          tc::tmem_ld16(tmem + tl + L::TY + 64 * hf + 32 * half, u[0]);
          tc::tmem_ld16(tmem + tl + L::TY + 64 * hf + 32 * half + 16, u[1]);
          tc::tmem_wait_ld();
          if (half == 1) {
            tc::fence_before_sync();
            tc::mbar_arrive(y_free);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t at = xo + tc::sw128(i, 4 * half + m);
            float xv[8], zv[8], f[8];
            widen<__nv_bfloat16>(lds_v4(smem, at), xv);
            widen<__nv_bfloat16>(z[4 * half + m], zv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[e] = fmaf(sg, __uint_as_float(u[m / 2][m % 2 * 8 + e]), skip * xv[e]);
              if (zg != nullptr) f[e] *= zv[e] * sigmoid_f(zv[e]);
            }
            const uint4 v = narrow<__nv_bfloat16>(f);
            if (whole) *reinterpret_cast<uint4*>(smem + at) = v;
            else if (live && lt < seg_n)
              *reinterpret_cast<uint4*>(og + static_cast<long>(c) * kC * a.H * P + 32 * half + 8 * m) = v;
          }
        }
        if (whole) tc::fence_async_smem();
        tc::mbar_arrive(staged + 8 * s);
      }
      if (!ok) *s_abort = 1;
    }
  } else if (warp < (kRows + kStates) / 32) {
    // ============================================================ states
    tc::regs_inc<kRegsStates>();
    constexpr int HN = N / 2;               // columns n of a thread
    const int half = (warp - kRows / 32) >> 2;
    const int p = 32 * q4 + lane;           // column of the x tile = TMEM lane
    const int k = NH == 2 ? q4 >> 1 : 0;    // its head
    const int pl = NH == 2 ? p & 63 : p;
    const bool live = k < nh;
    const int head = h0 + min(k, nh - 1), n0 = half * HN;
    const long dh = static_cast<long>(doc) * a.H + head;
    float h[HN];
#pragma unroll
    for (int e = 0; e < HN; ++e) h[e] = 0.f;
    if constexpr (READ) {
      if (a.S0 != nullptr) {
#pragma unroll
        for (int e = 0; e < HN; ++e) h[e] = a.S0[dh * (N * P) + (n0 + e) * P + pl];
      }
      if (seg > 0) tc::grid_dep_wait();
#pragma unroll 1
      for (int j = 0; j < seg; ++j) {
        const float* const rec = a.ws + (dh * (a.nseg - 1) + j) * kRec;
        const float keep = __ldcg(rec + N * P);
#pragma unroll
        for (int e = 0; e < HN; ++e) h[e] = fmaf(keep, h[e], __ldcg(rec + (n0 + e) * P + pl));
      }
    }
    // the bf16 copy [columns p][N] that C h^T reads
    const auto publish = [&]() {
      if constexpr (READ) {
#pragma unroll
        for (int m = 0; m < HN / 8; ++m) {
          const int col = n0 + 8 * m;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = h[8 * m + e];
          *reinterpret_cast<uint4*>(smem + L::H + col / 64 * 16384 + tc::sw128(p, col % 64 / 8)) = narrow<__nv_bfloat16>(f);
        }
        tc::fence_async_smem();
        tc::mbar_arrive(h_ready);
      }
    };
    float keep = 1.f, log_all = 0.f;
    // h takes the increment of the chunk before
    const auto update = [&](int c) {
      const int ok = wait(inc_done, c & 1);
      if (__any_sync(0xffffffffu, !ok)) return false;
      tc::fence_after_sync();
#pragma unroll
      for (int m = 0; m < HN / 16; ++m) {
        uint32_t u[16];
        tc::tmem_ld16(tmem + tl + L::TI + n0 + 16 * m, u);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) h[16 * m + e] = fmaf(keep, h[16 * m + e], __uint_as_float(u[e]));
      }
      return true;
    };
    publish();
    bool ok = true;
    for (int c = 0; c < nchunks; ++c) {
      const int s = c & 1, ph = (c >> 1) & 1;
      if (c > 0) {
        ok = update(c - 1);
        if (!ok) break;
        publish();
      }
      ok = wait(tab_full + 8 * s, ph) && wait(x_full + 8 * s, ph);
      if (__any_sync(0xffffffffu, !ok)) {
        ok = false;
        break;
      }
      const float* const sums = table(c, 0, k);
      float bs[4];
#pragma unroll
      for (int J = 0; J < 4; ++J) bs[J] = sums[32 * J + 31];
      const float all = between(bs, 0, 4);
      keep = ex2(all);
      log_all += all;
      const uint32_t xo = L::X + s * L::XT + (p >> 6) * 16384 + (p & 7) * 2;
      const int pc = (p & 63) >> 3;
#pragma unroll
      for (int b = 0; b < 4; ++b) {  // 16 tokens: one K step of the product
        const int t0 = 64 * half + 16 * b;
        const float after = ex2(between(bs, t0 / 32 + 1, 4));
        const float* const f = table(c, 2, k) + t0;
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 w4 = *reinterpret_cast<const float4*>(f + e);
          const float w[4] = {w4.x, w4.y, w4.z, w4.w};
          float v[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int t = t0 + e + d;
            const uint16_t raw = *reinterpret_cast<const uint16_t*>(smem + xo + t * 128 + ((pc ^ (t & 7)) << 4));
            v[d] = __uint_as_float(static_cast<uint32_t>(raw) << 16) * (w[d] * after);
          }
#pragma unroll
          for (int d = 0; d < 4; d += 2) {
            const uint32_t top = tc::pack_bf16x2(v[d], v[d + 1]);
            hi[(e + d) / 2] = top;
            lo[(e + d) / 2] = tc::pack_bf16x2(v[d] - __uint_as_float(top << 16), v[d + 1] - __uint_as_float(top & 0xffff0000u));
          }
        }
        tc::tmem_st8(tmem + tl + L::TX + t0 / 2, hi);
        tc::tmem_st8(tmem + tl + L::TX + 64 + t0 / 2, lo);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(xw_ready);
      tc::mbar_arrive(tab_free + 8 * s);
    }
    if (ok && nchunks > 0) ok = update(nchunks - 1);
    if (!ok) *s_abort = 1;
    if (ok && live) {
      float* dst = nullptr;
      if (!READ) {
        dst = a.ws + (dh * (a.nseg - 1) + seg) * kRec;
        if (half == 0 && pl == 0) __stcg(dst + N * P, ex2(log_all));
      } else if (seg == segs - 1 && a.S_final != nullptr) {
        dst = a.S_final + dh * (N * P);
      }
      if (dst != nullptr) {
#pragma unroll
        for (int e = 0; e < HN; ++e) __stcg(dst + (n0 + e) * P + pl, h[e]);
      }
    }
  } else {
    tc::regs_dec<kRegsRest>();  // one call site for the whole warpgroup
    if (warp == kWarpIssue) {
      // ========================================================== MMA issue (one thread)
      if (lane == 0) {
        constexpr uint32_t kIdTile = tc::idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdInc = tc::idesc_bf16(128, N, false, true);
        constexpr uint32_t kIdY = tc::idesc_bf16(128, P, false, true);
        bool ok = true;
        for (int c = 0; c < nchunks; ++c) {
          const int s = c & 1, ph = (c >> 1) & 1;
          const uint64_t d_c = tc::desc_sw128(base + L::C, 16, 1024), d_h = tc::desc_sw128(base + L::H, 16, 1024);
          const uint64_t d_bk = tc::desc_sw128(base + L::B + s * L::NT, 16, 1024);
          const uint64_t d_bm = tc::desc_sw128(base + L::B + s * L::NT, 16384, 1024);
          const uint64_t d_x = tc::desc_sw128(base + L::X + s * L::XT, 16384, 1024);
          ok = wait(b_full + 8 * s, ph);
          if constexpr (READ) {
            ok = ok && wait(c_full, c & 1) && wait(x_full + 8 * s, ph);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int k = 0; k < N / 16; ++k) {
              const uint64_t ko = static_cast<uint64_t>((k / 4) * 1024 + (k % 4) * 2);
              tc::mma_bf16(tmem + L::TG, d_c + ko, d_bk + ko, kIdTile, k > 0);
            }
            tc::mma_commit(g_done);
            ok = wait(h_ready, c & 1) && (c == 0 || wait(y_free, (c - 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int k = 0; k < N / 16; ++k) {
              const uint64_t ko = static_cast<uint64_t>((k / 4) * 1024 + (k % 4) * 2);
              tc::mma_bf16(tmem + L::TY, d_c + ko, d_h + ko, kIdTile, k > 0);
            }
            tc::mma_commit(yoff_done);
          }
          ok = ok && wait(xw_ready, c & 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int k = 0; k < 16; ++k)  // the high parts of the 128 tokens, then the low ones
            tc::mma_bf16_ta(tmem + L::TI, tmem + L::TX + 8 * k, d_bm + static_cast<uint64_t>(k & 7) * 128, kIdInc, k > 0);
          tc::mma_commit(inc_done);
          if constexpr (READ) {
            ok = wait(m_ready, c & 1);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int hh = 0; hh < nh; ++hh)
#pragma unroll 1
              for (int k = 0; k < kC / 16; ++k)
                tc::mma_bf16_ta(tmem + L::TY + 64 * hh, tmem + L::TG + 32 * (k / 2) + 16 * hh + 8 * (k % 2),
                                d_x + static_cast<uint64_t>(hh) * 1024 + static_cast<uint64_t>(k) * 128, kIdY, 1u);
            tc::mma_commit(y_done);
          }
        }
        if (!ok) *s_abort = 1;
        // no product is under way when TMEM and the tiles are given up
        tc::mma_commit(drain);
        tc::mbar_wait(drain, 0, kWaitCycles);
      }
    } else if (warp == kWarpTma) {
      // ========================================================== loads and stores (one thread)
      if (lane == 0) {
        const int xc = h0 * P, nc = g * N, row = static_cast<int>(row0);
        const uint32_t xbytes = (NH == 1 ? 2 : nh) * 16384u;
        const auto load_x = [&](int c) {
          tc::mbar_arrive_expect_tx(x_full + 8 * (c & 1), xbytes);
          for (uint32_t j = 0; j < xbytes / 16384; ++j)
            tc::tma_load_3d(base + L::X + (c & 1) * L::XT + j * 16384, &maps.x, xc + 64 * j, 0, row + c * kC,
                            x_full + 8 * (c & 1));
        };
        const auto load_b = [&](int c) {
          tc::mbar_arrive_expect_tx(b_full + 8 * (c & 1), L::NT);
          for (int j = 0; j < N / 64; ++j)
            tc::tma_load_3d(base + L::B + (c & 1) * L::NT + j * 16384, &maps.b, nc + 64 * j, 0, row + c * kC,
                            b_full + 8 * (c & 1));
        };
        const auto load_c = [&](int c) {
          if constexpr (READ) {
            tc::mbar_arrive_expect_tx(c_full, L::NT);
            for (int j = 0; j < N / 64; ++j)
              tc::tma_load_3d(base + L::C + j * 16384, &maps.c, nc + 64 * j, 0, row + c * kC, c_full);
          }
        };
        int nx = 0, nb = 0, ncl = 0;  // loads issued
        for (; nb < 2 && nb < nchunks; ++nb, ++nx) {
          load_b(nb);
          load_x(nb);
        }
        if (nchunks > 0 && READ) load_c(ncl++);
        bool ok = true;
        for (int c = 0; c < nchunks && ok; ++c) {
          const int s = c & 1, ph = (c >> 1) & 1;
          if constexpr (READ) {
            ok = wait(yoff_done, c & 1);
            if (!ok) break;
            if (c + 1 < nchunks) load_c(ncl++);
          }
          ok = wait(inc_done, c & 1);
          if (!ok) break;
          if (c + 2 < nchunks) load_b(nb++);
          if constexpr (READ) {
            ok = wait(staged + 8 * s, ph);
            if (!ok) break;
            if (c * kC + kC <= seg_n) {  // a whole chunk was staged
              for (uint32_t j = 0; j < xbytes / 16384; ++j)
                tc::tma_store_3d(&maps.out, base + L::X + s * L::XT + j * 16384, xc + 64 * j, 0, row + c * kC);
              tc::bulk_commit();
              tc::bulk_wait_read0();  // the buffer may be refilled once the store has read it
            }
          }
          if (c + 2 < nchunks) load_x(nx++);  // (without reading: xw came before the increment)
        }
        if (!ok) *s_abort = 1;
        tc::bulk_wait0();
        if (*s_abort) {  // no copy is under way when the tiles are given up: the last load of each buffer
          for (int i = 0; i < 2; ++i) {
            if (nx > i) tc::mbar_wait(x_full + 8 * i, ((nx - 1 - i) >> 1) & 1, kWaitCycles);
            if (nb > i) tc::mbar_wait(b_full + 8 * i, ((nb - 1 - i) >> 1) & 1, kWaitCycles);
          }
          if (ncl > 0) tc::mbar_wait(c_full, (ncl - 1) & 1, kWaitCycles);
        }
      }
    } else if (warp - kWarpTab < NH) {
      // ========================================================== step sizes and decays of a head
      const int k = warp - kWarpTab, head = h0 + min(k, nh - 1);
      const float bias = a.dt_bias != nullptr ? a.dt_bias[head] : 0.f, A2 = a.A[head] * kLog2e;
      const __nv_bfloat16* const src = static_cast<const __nv_bfloat16*>(a.dt) + row0 * a.dts + head;
      float raw[4];
      const auto load = [&](int c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = c * kC + 4 * lane + e;
          raw[e] = t < seg_n ? to_f(src[t * a.dts]) : 0.f;
        }
      };
      load(0);
      bool ok = true;
      for (int c = 0; c < nchunks; ++c) {
        const int s = c & 1;
        float d[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[e] = c * kC + 4 * lane + e < seg_n ? step_size(raw[e], bias, a.softplus) : 0.f;
          l[e] = fmaxf(d[e] * A2, kLeastLog);
        }
        load(c + 1);
        // sums inside the block of 32 tokens (8 lanes): p up to a token, t behind it
        float p[4], t[4];
        p[0] = l[0];
        t[3] = 0.f;
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          p[e] = p[e - 1] + l[e];
          t[3 - e] = t[4 - e] + l[4 - e];
        }
        float up = p[3], down = p[3];
#pragma unroll
        for (int o = 1; o < 8; o *= 2) {
          const float u = __shfl_up_sync(0xffffffffu, up, o, 8), v = __shfl_down_sync(0xffffffffu, down, o, 8);
          if ((lane & 7) >= o) up += u;
          if ((lane & 7) + o < 8) down += v;
        }
        const float left = __shfl_up_sync(0xffffffffu, up, 1, 8), right = __shfl_down_sync(0xffffffffu, down, 1, 8);
        const float before = (lane & 7) > 0 ? left : 0.f, behind = (lane & 7) < 7 ? right : 0.f;
        if (c >= 2) ok = wait(tab_free + 8 * s, ((c >> 1) + 1) & 1);
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        float q[4], f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] += before;
          q[e] = p[e] - lg2(d[e]);  // a step of 0: infinity, whose e^- is 0
          f[e] = ex2(t[e] + behind) * d[e];
        }
        float* const dst = reinterpret_cast<float*>(smem + L::TAB + s * L::TAB1) + k * kC + 4 * lane;
        *reinterpret_cast<float4*>(dst) = make_float4(p[0], p[1], p[2], p[3]);
        *reinterpret_cast<float4*>(dst + 2 * kC) = make_float4(q[0], q[1], q[2], q[3]);
        *reinterpret_cast<float4*>(dst + 4 * kC) = make_float4(f[0], f[1], f[2], f[3]);
        tc::mbar_arrive(tab_full + 8 * s);
      }
      if (!ok) *s_abort = 1;
    }
  }

  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (*s_abort && tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, kDevInternal);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// [rows, cols] with `stride` elements from row to row: boxes of 64 columns x 128 rows.
cudaError_t make_map(CUtensorMap* map, const void* base, long rows, long cols, long stride) {
  const uint64_t dims[3] = {static_cast<uint64_t>(cols), 1, static_cast<uint64_t>(rows)};
  const uint64_t strides[2] = {static_cast<uint64_t>(stride) * 2, static_cast<uint64_t>(stride) * 2};
  const uint32_t box[3] = {64, 1, kC};
  return encode_bf16_map(map, base, 3, dims, strides, box);
}

template <int P, int N, bool READ>
cudaError_t go(const SsmArgs& a, const Maps& maps, bool dependent, cudaStream_t stream) {
  constexpr int NH = P == 64 ? 2 : 1;
  static std::atomic<unsigned long long> configured{0};  // bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !((configured.load(std::memory_order_relaxed) >> dev) & 1ull))) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<P, N, READ>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::BYTES);
    if (e == cudaSuccess && dev < 64) configured.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  const int R = a.H / a.G;
  const long grid = static_cast<long>(a.docs.n_docs) * a.G * ((R + NH - 1) / NH) * (READ ? a.nseg : a.nseg - 1);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Lay<N>::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;  // the scan behind its own kernel A alone: it must not overlap anything else
  e = cudaLaunchKernelEx(&cfg, ssm_tc_kernel<P, N, READ>, a, maps);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int P, int N>
cudaError_t both(const SsmArgs& a, cudaStream_t stream) {
  Maps maps;
  memset(&maps, 0, sizeof(maps));  // no rows: the kernels issue no copy
  const long rows = a.docs.total_rows, wide = static_cast<long>(a.H) * P, narrow = static_cast<long>(a.G) * N;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = make_map(&maps.x, a.x, rows, wide, a.xs);
    if (e == cudaSuccess) e = make_map(&maps.b, a.B, rows, narrow, a.bs);
    if (e == cudaSuccess) e = make_map(&maps.c, a.C, rows, narrow, a.cs);
    if (e == cudaSuccess) e = make_map(&maps.out, a.out, rows, wide, wide);
  }
  if (e == cudaSuccess && a.nseg > 1) e = go<P, N, false>(a, maps, false, stream);
  return e != cudaSuccess ? e : go<P, N, true>(a, maps, a.nseg > 1, stream);
}

}  // namespace

bool ssm_tc_supported(DType dt, int P, int N) {
  return dt == DType::BF16 && (P == 64 || P == 128) && (N == 64 || N == 128);
}

// Segments of a document, by an estimate in units of one chunk of the scan: waves of one CTA an SM, each its chunks
// and 1.5 of set-up; kernel A's chunks cost 0.6. A longer plan has to be 5 % faster.
SsmPlan ssm_plan_tc(const SsmArgs& a) {
  const int NH = a.P == 64 ? 2 : 1, R = a.H / a.G;
  const long units = static_cast<long>(a.G) * ((R + NH - 1) / NH);
  const long docs = a.docs.n_docs, longest = std::max(1, (a.docs.max_seqlen + kC - 1) / kC);
  const double mean = std::max(1.0, static_cast<double>(a.docs.total_rows) / kC / docs);  // chunks of a document
  SsmPlan best{};
  double best_cost = 1e300;
  for (long len = longest; len >= 1; --len) {
    const long nseg = (longest + len - 1) / len;
    if (nseg > 64) break;
    const double per_doc = std::max(1.0, std::min(static_cast<double>(nseg), mean / static_cast<double>(len)));
    const auto waves = [](double ctas) { return static_cast<double>(static_cast<long>((ctas + 151.0) / 152.0)); };
    double cost = waves(units * docs * per_doc) * (len + 1.5);
    if (nseg > 1) cost += waves(units * docs * std::max(1.0, per_doc - 1)) * (0.6 * len + 1.5);
    if (cost < 0.95 * best_cost) {
      best_cost = cost;
      best.nseg = static_cast<int>(nseg);
      best.seg_len = static_cast<int>(len) * kC;
    }
  }
  best.ws_bytes = static_cast<size_t>(docs) * a.H * (best.nseg - 1) * (static_cast<size_t>(a.N) * a.P + kSsmRecTail) * 4;
  return best;
}

cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t stream) {
  if (a.P == 64) return a.N == 64 ? both<64, 64>(a, stream) : both<64, 128>(a, stream);
  return a.N == 64 ? both<128, 64>(a, stream) : both<128, 128>(a, stream);
}

}  // namespace rapt
