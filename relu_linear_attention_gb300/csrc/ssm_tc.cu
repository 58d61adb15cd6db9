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
// 2^-64 for 0. Two bf16 parts of xw keep the fp32 state to 1.5 x 2^-15 of its terms (the weight's second part is off by
// 2^-16 of it, the sum that makes the low part by 2^-15; 16 M random pairs: 2^-14.9): with one part it would be 2^-7,
// and the state is an output and the start of everything later. For a third part TMEM has no room at N = 128 (all 512
// columns: G, xw, the increment, Y). B and x enter exactly as they are.
//
// Decays are formed from sums inside blocks of 32 tokens, so that a difference of logarithms is that of sums of at
// most 32 and what lies between: left of the diagonal block, e^(s_i - s_j) = e^(s_i - s at the end of j's block) x
// e^(that - s_j), one factor a row and block and one a column, both at most 1: no exponential an element, no
// overflow at any decay. On the diagonal block each element has its own. a_t stops at -160 log 2 (2^-160 is 0).
//
// Warps (896 threads, one CTA an SM):
//   0-7   rows:   step sizes, decays and their sums, a thread a head and token; G -> M, a TMEM lane quarter and every
//                 other 16 keys each;
//   8-15  states: the increment into h (fp32, in registers) and its bf16 copy in shared memory, then xw of half of the
//                 next chunk's tokens (a TMEM lane is a column of x);
//   16-23 ends:   the epilogue of one half of Y (64 columns) after the other, a lane quarter and 32 columns each: Y is
//                 free for the next chunk's products as soon as it is in registers; y goes where x was in shared
//                 memory, from where the TMA stores it, and z comes by TMA, half a tile at a time (rows of 64 bytes by
//                 plain loads and stores kept the load-store unit busy for half of the time);
//   24    MMA issue, 25 TMA of B and C, 26 of x and the output, 27 of z.
// Shared memory: two x and two B tiles, one C tile, the state copy, half a tile of gates, the decay tables. A document
// is cut into segments where there are fewer units than SMs; kernel A (the same code without reading) gives their
// increments.
// Every wait is bounded; one that gives up sets RAPT_DEV_INTERNAL and the CTA winds down.
//
// 4 x 4096 tokens x 64 heads of 64, N = 128: 146 us (the bytes alone 62, the products 47); 65536 packed tokens x 32
// heads of 64, N = 64: 263 us; 32768 tokens x 16 heads of 128, N = 128: 177 us in segments. What bounds it is a
// chunk's chain, 9 thousand cycles: the state and its copy wait for the increment, the rows for G, the epilogue for
// Y, one after the other; the tensor pipe is busy for a third of it and the issue slots for half.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "ssm.cuh"
#include "tc_features.cuh"
#include "tc_utils.cuh"
#include "tensor_map.h"

namespace rapt {
namespace {

using namespace ssm;

constexpr int kC = 128;                       // tokens of a chunk
constexpr int kRows = 256, kStates = 256, kEnds = 256;  // threads of the groups
constexpr int kThreads = kRows + kStates + kEnds + 128;
constexpr int kWarpIssue = (kRows + kStates + kEnds) / 32, kWarpLoad = kWarpIssue + 1, kWarpX = kWarpIssue + 2, kWarpZ = kWarpIssue + 3;
constexpr long long kWaitCycles = 1000000000LL;  // ~0.5 s: what is not done by then never will be
constexpr uint32_t kDevInternal = 2u;
// Registers: kernel A has no epilogue, and the states of N = 128 want more than 96 (spilled, its increments take 10 % longer).
constexpr int kLaunchRegs = 72, kRegsRows = 56, kRegsRest = 40;
template <bool READ>
constexpr int kRegsStates = READ ? 96 : 128;
template <bool READ>
constexpr int kRegsEnds = READ ? 80 : 24;
template <bool READ>
constexpr int kRegsSum =
    kRows * kRegsRows + kStates * kRegsStates<READ> + kEnds * kRegsEnds<READ> + 128 * kRegsRest;
static_assert(kRegsSum<true> <= kThreads * kLaunchRegs && kRegsSum<false> <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kBarRows = 1, kBarStates = 2, kBarEnds = 3;  // named barriers of the groups
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeastLog = -160.f;  // of a token's decay, base 2
constexpr float kLeastRow = -64.f;   // of a row's common factor

// Byte offsets from a 1024-byte aligned base, and TMEM columns.
template <int N>
struct Lay {
  static constexpr uint32_t XT = 32768, NT = N / 64 * 16384;
  static constexpr uint32_t X = 0, B = 2 * XT, C = B + 2 * NT, H = C + NT;
  static constexpr uint32_t Z = H + NT;  // the gates of half a tile's columns
  static constexpr uint32_t TAB = Z + 16384;  // [2 buffers]: [p, q, f][2 heads][kC] fp32, [2 parts of w][2 heads][kC] bf16
  static constexpr uint32_t TABW = 3 * 2 * kC * 4, TAB1 = TABW + 2 * 2 * kC * 2;
  static constexpr uint32_t MASK = TAB + 2 * TAB1;  // [4][32 lanes][4]: bf16 pairs of keys that a lane's row sees
  static constexpr uint32_t SUMS = MASK + 2048;  // [2 buffers][2 heads][4 blocks]: log2 of the blocks' decays
  static constexpr uint32_t BAR = SUMS + 64;
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
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two bf16 values as floats.
__device__ __forceinline__ float2 widen2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 v) { return tc::pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ uint4 lds_v4(const uint8_t* sm, uint32_t off) { return *reinterpret_cast<const uint4*>(sm + off); }

// Products issued by a converged warp, one elected lane each: the operands stay in uniform registers. (In a branch
// of one lane a product took 160 cycles to issue in a loop, 64 unrolled; N = 64 from TMEM 48 unrolled, 33 so.)
// Descriptors are given by their low words; the high one is that of every swizzled tile (8-row groups 1024 bytes
// apart, version 1, 128-byte swizzle).
constexpr uint32_t kDescHigh = 64u | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16;
}
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n mov.b64 x, {%1, %5};\n mov.b64 y, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ta(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n mov.b64 y, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}

// One probe of a phase, which may suspend the thread for as long as the hardware likes. (With a time of 20 us to
// suspend for, the probe becomes a loop of short sleeps: waits then noticed a phase up to 1000 cycles late, and
// polling took a third of the issue slots; the scan of 16384 tokens x 64 heads: 193 us.)
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for a phase; false where that gives up, or the CTA has.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const volatile int* abort) {
  if (probe(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  for (int i = 1;; ++i) {
    if (probe(bar, parity)) return true;
    if ((i & 63) == 0 && ((abort != nullptr && *abort != 0) || clock64() - t0 > kWaitCycles)) return false;
  }
}
// Registers of a thread from here on.
template <int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (N > kLaunchRegs) tc::regs_inc<N>();
  if constexpr (N < kLaunchRegs) tc::regs_dec<N>();
}
// 16 lanes x 16 columns: thread t's value r[2 i + u] goes to lane 8 u + t / 4 and column 4 i + t % 4, which is how a
// transposing ldmatrix of 8 x 8 bf16 hands out pairs of rows.
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// log2 sg_i of row i of lane quarter q4, from a head's sums p inside blocks of 32.
__device__ __forceinline__ float row_log(const float* p, int i, int q4) {
  float all = p[i];
#pragma unroll
  for (int J = 0; J < 3; ++J) all += J < q4 ? p[32 * J + 31] : 0.f;
  return fmaxf(all, kLeastRow);
}

// f times z sigmoid(z) of 8 bf16 values z, that product first: f z may overflow where sigmoid(z) is 0. (One reciprocal
// for four, 1 / (a b c d) times the others' products, costs more instructions than it saves.)
__device__ __forceinline__ void gate_by(const uint4& z4, float2 (&f)[4]) {
  const uint32_t w[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 z = widen2(w[e]), x = __fmul2_rn(z, make_float2(-kLog2e, -kLog2e));
    const float2 d = __fadd2_rn(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
    f[e] = __fmul2_rn(f[e], __fmul2_rn(z, r));
  }
}

struct Maps {
  CUtensorMap x, b, c, z, out;
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
  const int halves = NH == 2 ? nh : 2;     // of the tile's columns
  long row0;
  int n;
  const bool good = doc_rows(a.docs, doc, row0, n);
  if (READ && !good && seg == 0 && unit == 0 && tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, 1u);
  const int segs = n > 0 ? (n + a.seg_len - 1) / a.seg_len : 1;
  if (!good || seg >= (READ ? segs : segs - 1)) {  // uniform across the CTA, before any allocation
    if (READ) end_behind_records(a);
    return;
  }
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
  const uint32_t inc_done = bars + 104, yoff_done = bars + 112, drain = bars + 120, staged = bars + 128;
  const uint32_t y_done = bars + 144, y_free = bars + 160, z_full = bars + 176, z_free = bars + 184;
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
      tc::mbar_init(tab_full + 8 * i, kRows);
      tc::mbar_init(tab_free + 8 * i, READ ? kStates + kEnds : kStates);
      tc::mbar_init(staged + 8 * i, kEnds);
      tc::mbar_init(y_done + 8 * i, 1);
      tc::mbar_init(y_free + 8 * i, kEnds);
    }
    tc::mbar_init(c_full, 1);
    tc::mbar_init(g_done, 1);
    tc::mbar_init(m_ready, kRows);
    tc::mbar_init(h_ready, kStates);
    tc::mbar_init(xw_ready, kStates);
    tc::mbar_init(inc_done, 1);
    tc::mbar_init(yoff_done, 1);
    tc::mbar_init(drain, 1);
    tc::mbar_init(z_full, 1);
    tc::mbar_init(z_free, kEnds);
    tc::mbar_fence_init();
    *s_abort = 0;
  }
  if (READ && tid < 512) {  // pair e of keys (2 e, 2 e + 1) for the row of this lane
    const int l = tid / 4 % 32, e = tid / 128 * 4 + tid % 4;
    reinterpret_cast<uint32_t*>(smem + L::MASK)[tid] = 2 * e + 1 <= l ? 0xffffffffu : 2 * e <= l ? 0x0000ffffu : 0u;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const auto wait = [&](uint32_t bar, int parity) { return wait_phase(bar, parity, s_abort); };
  // A group of warps: its first one waits, the others at a barrier, where they take no issue slots from those that
  // compute. False for all of them where the wait gave up.
  const auto group = [&](uint32_t id, uint32_t threads, bool leader, uint32_t b0, int p0, uint32_t b1, int p1, uint32_t b2, int p2) {
    int bad = 0;
    if (leader) bad = !(wait(b0, p0) && (b1 == 0 || wait(b1, p1)) && (b2 == 0 || wait(b2, p2)));
    return feat::group_sync_or(id, threads, bad) == 0;
  };
  // for what is under way, whether or not the CTA has given up
  const auto last = [&](uint32_t bar, int parity) { wait_phase(bar, parity, nullptr); };
  const auto table = [&](int c, int which, int head) {
    return reinterpret_cast<const float*>(smem + L::TAB + (c & 1) * L::TAB1) + (which * 2 + head) * kC;
  };
  const int q4 = warp & 3;  // TMEM lane quarter
  const uint32_t tl = static_cast<uint32_t>(32 * q4) << 16;

  if (warp < kRows / 32) {
    // ============================================================ rows
    set_regs<kRegsRows>();
    // The tables of a chunk: thread (head, token), a warp a block of 32 tokens.
    const int tk = warp >> 2;
    const bool tables_mine = tk < NH;
    const __nv_bfloat16* const dts = static_cast<const __nv_bfloat16*>(a.dt) + row0 * a.dts + h0 + min(tk, nh - 1);
    const float bias = a.dt_bias != nullptr ? a.dt_bias[h0 + min(tk, nh - 1)] : 0.f, A2 = a.A[h0 + min(tk, nh - 1)] * kLog2e;
    const auto load_dt = [&](int c) -> uint16_t {  // (as it is: a conversion would wait for it here)
      const int t = c * kC + 32 * q4 + lane;
      return tables_mine && t < seg_n ? __ldg(reinterpret_cast<const uint16_t*>(dts) + static_cast<long>(t) * a.dts)
                                      : static_cast<uint16_t>(0);
    };
    uint16_t raw0 = load_dt(0), raw1 = load_dt(1);  // of the next chunk and the one behind it
    const auto tables = [&](int c) {
      const int s = c & 1, t = 32 * q4 + lane;
      const float d = c * kC + t < seg_n 
                          ? step_size(__uint_as_float(static_cast<uint32_t>(raw0) << 16), bias, a.softplus)
                          : 0.f;
      // (a NaN stays one; behind the document's end the state is kept, whatever A)
      const float l = c * kC + t < seg_n ? max_nan(d * A2, kLeastLog) : 0.f;
      raw0 = raw1;
      raw1 = load_dt(c + 2);
      // sums inside the block: p up to a token, behind it u
      float p = l, u = l;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float x = __shfl_up_sync(0xffffffffu, p, o), y = __shfl_down_sync(0xffffffffu, u, o);
        if (lane >= o) p += x;
        if (lane + o < 32) u += y;
      }
      const float sum = __shfl_sync(0xffffffffu, p, 31), next = __shfl_down_sync(0xffffffffu, u, 1);
      u = lane < 31 ? next : 0.f;
      // the buffer's last readers are done
      if (c >= 2 && !group(kBarRows, kRows, warp == 0, tab_free + 8 * s, ((c >> 1) + 1) & 1, 0, 0, 0, 0)) return false;
      float* const sums = reinterpret_cast<float*>(smem + L::SUMS) + 8 * s;
      if (lane == 0) sums[4 * tk + q4] = sum;
      tc::named_sync(kBarRows, kRows);
      if (tables_mine) {
        const float b1 = sums[4 * tk + 1], b2 = sums[4 * tk + 2], b3 = sums[4 * tk + 3];
        const float f = ex2(u) * d;
        const float w = f * ex2(q4 == 0 ? b1 + b2 + b3 : q4 == 1 ? b2 + b3 : q4 == 2 ? b3 : 0.f);
        float* const dst = reinterpret_cast<float*>(smem + L::TAB + s * L::TAB1) + tk * kC + t;
        dst[0] = p;
        dst[2 * kC] = p - lg2(d);  // a step of 0: infinity, whose e^- is 0
        dst[4 * kC] = f;
        __nv_bfloat16* const dw = reinterpret_cast<__nv_bfloat16*>(smem + L::TAB + s * L::TAB1 + L::TABW) + tk * kC + t;
        const __nv_bfloat16 w1 = __float2bfloat16_rn(w);
        dw[0] = w1;
        dw[2 * kC] = __float2bfloat16_rn(w - __bfloat162float(w1));
      }
      tc::mbar_arrive(tab_full + 8 * s);
      return true;
    };
    bool ok = nchunks == 0 || tables(0);
    if constexpr (READ) {
      const int i = 32 * q4 + lane;
      for (int c = 0; c < nchunks; ++c) {
        ok = group(kBarRows, kRows, warp == 0, g_done, c & 1, 0, 0, 0, 0);
        if (!ok) break;
        tc::fence_after_sync();
        float pl[NH], far[NH];  // this row's p_i - log2 sg_i for each head; the same and the blocks up to the keys'
#pragma unroll
        for (int k = 0; k < NH; ++k) {
          const float* const p = table(c, 0, k);
          pl[k] = far[k] = p[i] - row_log(p, i, q4);
        }
        // 16 keys of every block: their G makes room for the M of both heads
#pragma unroll 1
        for (int J = 3; J >= 0; --J) {
          const int k0 = 32 * J + 16 * (warp >> 2);
          const uint32_t tg = tmem + tl + L::TG + k0;
          uint32_t w[NH][8];
          if (J > q4) {
#pragma unroll
            for (int k = 0; k < NH; ++k)
#pragma unroll
              for (int e = 0; e < 8; ++e) w[k][e] = 0u;
          } else {
            uint32_t u[16];
            tc::tmem_ld16(tg, u);
            tc::tmem_wait_ld();
            const auto val2 = [&](int e) { return make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])); };
            if (J == q4) {
#pragma unroll
              for (int k = 0; k < NH; ++k) {
                const float* const q = table(c, 1, k) + k0;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 v = *reinterpret_cast<const float4*>(q + e);
                  w[k][e / 2] = pack2(__fmul2_rn(val2(e), make_float2(ex2(pl[k] - v.x), ex2(pl[k] - v.y))));
                  w[k][e / 2 + 1] = pack2(__fmul2_rn(val2(e + 2), make_float2(ex2(pl[k] - v.z), ex2(pl[k] - v.w))));
                }
              }
#pragma unroll
              for (int e = 0; e < 8; e += 4) {  // keys behind the row's token: nothing, whatever came out
                const uint4 keep = lds_v4(smem, L::MASK + (2 * (warp >> 2) + e / 4) * 512 + lane * 16);
#pragma unroll
                for (int k = 0; k < NH; ++k)
                  w[k][e] &= keep.x, w[k][e + 1] &= keep.y, w[k][e + 2] &= keep.z, w[k][e + 3] &= keep.w;
              }
            } else {
#pragma unroll
              for (int k = 0; k < NH; ++k) {
                const float* const f = table(c, 2, k) + k0;
                const float rf = ex2(far[k]);
                const float2 r2 = make_float2(rf, rf);
                far[k] += table(c, 0, k)[32 * J + 31];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                  const float4 v = *reinterpret_cast<const float4*>(f + e);
                  w[k][e / 2] = pack2(__fmul2_rn(val2(e), __fmul2_rn(r2, make_float2(v.x, v.y))));
                  w[k][e / 2 + 1] = pack2(__fmul2_rn(val2(e + 2), __fmul2_rn(r2, make_float2(v.z, v.w))));
                }
              }
            }
          }
#pragma unroll
          for (int k = 0; k < NH; ++k) tc::tmem_st8(tg + 8 * k, w[k]);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(m_ready);
        if (c + 1 < nchunks) ok = ok && tables(c + 1);
        if (!ok) break;
      }
    } else {
      for (int c = 1; c < nchunks && ok; ++c) ok = tables(c);
    }
    if (!ok) *s_abort = 1;
  } else if (warp < (kRows + kStates) / 32) {
    // ============================================================ states
    set_regs<kRegsStates<READ>>();
    constexpr int HN = N / 2;               // columns n of a thread
    const int half = (warp - kRows / 32) >> 2;
    const int p = 32 * q4 + lane;           // column of the x tile = TMEM lane
    const int k = NH == 2 ? q4 >> 1 : 0;    // its head
    const int pl = NH == 2 ? p & 63 : p;
    const bool live = k < nh;
    const int head = h0 + min(k, nh - 1), n0 = half * HN;
    const long dh = static_cast<long>(doc) * a.H + head;
    float2 h[HN / 2];
#pragma unroll
    for (int e = 0; e < HN / 2; ++e) h[e] = make_float2(0.f, 0.f);
    if constexpr (READ) {
      // (a segment's record holds the state at its end by now)
      const float* const from = seg > 0 ? a.ws + record(a, doc, row0 - seg_start, seg - 1, head) * kRec : a.S0 != nullptr ? a.S0 + dh * (N * P) : nullptr;
      if (seg > 0) tc::grid_dep_wait();
      if (from != nullptr) {
#pragma unroll
        for (int e = 0; e < HN / 2; ++e)
          h[e] = make_float2(__ldcg(from + (n0 + 2 * e) * P + pl), __ldcg(from + (n0 + 2 * e + 1) * P + pl));
      }
    }
    // the bf16 copy [columns p][N] that C h^T reads
    const auto publish = [&]() {
      if constexpr (READ) {
#pragma unroll
        for (int m = 0; m < HN / 8; ++m) {
          const int col = n0 + 8 * m;
          *reinterpret_cast<uint4*>(smem + L::H + col / 64 * 16384 + tc::sw128(p, col % 64 / 8)) =
              make_uint4(pack2(h[4 * m]), pack2(h[4 * m + 1]), pack2(h[4 * m + 2]), pack2(h[4 * m + 3]));
        }
        tc::fence_async_smem();
        tc::mbar_arrive(h_ready);
      }
    };
    float keep = 1.f, log_all = 0.f;
    // h takes the increment of the chunk before
    const auto update = [&](int c) {
      if (!group(kBarStates, kStates, warp == kRows / 32, inc_done, c & 1, 0, 0, 0, 0)) return false;
      tc::fence_after_sync();
#pragma unroll
      for (int m = 0; m < HN / 16; ++m) {
        uint32_t u[16];
        tc::tmem_ld16(tmem + tl + L::TI + n0 + 16 * m, u);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          h[8 * m + e / 2] = __ffma2_rn(make_float2(keep, keep), h[8 * m + e / 2],
                                        make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])));
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
        publish();  // (C h^T of the chunk before came ahead of its increment: its copy has been read)
      }
      const bool ragged = READ && c * kC + kC > seg_n;
      ok = group(kBarStates, kStates, warp == kRows / 32, tab_full + 8 * s, ph, x_full + 8 * s, ph, ragged ? g_done : 0u, c & 1);
      if (!ok) break;
      if (__builtin_expect(ragged, false)) {
        // The tiles go on with the next document's tokens, of weight 0: zeros in their place, as 0 times what is not
        // finite is no number. (G has been formed, so B has arrived and been read. A row is 128 bytes of each tile.
        // Fenced below, where the stores are long done: 11397 tokens in 120 documents, 92 heads of 64, N = 128: 419 us,
        // 427 with a wait and a fence of its own here, 413 without zeros.)
        uint8_t* const x = smem + L::X + s * L::XT;
        uint8_t* const b = smem + L::B + s * L::NT;
#pragma unroll 1
        for (int o = (seg_n - c * kC) * 128 + (tid - kRows) * 16; o < 16384; o += kStates * 16) {
          const uint4 none = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(x + o) = none;
          *reinterpret_cast<uint4*>(x + 16384 + o) = none;
          *reinterpret_cast<uint4*>(b + o) = none;
          if (N == 128) *reinterpret_cast<uint4*>(b + 16384 + o) = none;
        }
        tc::named_sync(kBarStates, kStates);
      }
      const float* const sums = table(c, 0, k);
      const float all = sums[31] + sums[63] + sums[95] + sums[127];
      keep = ex2(all);
      log_all += all;
      // xw of this warp's 32 columns and 64 tokens, two tokens a register as the product wants them: with the weight
      // in two bf16 parts, w = w1 + w2, hi = bf16(x w1) leaves a remainder that bf16 holds exactly, and
      // lo = bf16(x w2 + (x w1 - hi)). Three instructions for two values.
      const uint32_t* const w1 = reinterpret_cast<const uint32_t*>(smem + L::TAB + s * L::TAB1 + L::TABW) + k * (kC / 2);
      const uint32_t* const w2 = w1 + kC;
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {  // 16 columns, 32 tokens
        const int c16 = 32 * q4 + 16 * (j & 1), t0 = 64 * half + 32 * (j >> 1);
        // 8 x 8 blocks (tokens t0 + 8 i, columns c16 + 8 u) in the order 2 i + u; this lane's row of one of them
        const int t = t0 + 8 * (lane >> 4) + (lane & 7), cc = c16 + (lane & 8);
        const uint32_t from =
            base + L::X + s * L::XT + (cc >> 6) * 16384 + t * 128 + ((((cc & 63) >> 3) ^ (lane & 7)) << 4);
        uint32_t x[8], hi[8];
        ldmatrix_trans(from, x[0], x[1], x[2], x[3]);
        ldmatrix_trans(from + 16 * 128, x[4], x[5], x[6], x[7]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = w1[t0 / 2 + 4 * i + (lane & 3)], b = w2[t0 / 2 + 4 * i + (lane & 3)];
#pragma unroll
          for (int u = 2 * i; u < 2 * i + 2; ++u) {
            hi[u] = mul_bf16x2(x[u], a);
            x[u] = fma_bf16x2(x[u], b, fma_bf16x2(x[u], a, hi[u] ^ 0x80008000u));
          }
        }
        const uint32_t to = tmem + tl + (static_cast<uint32_t>(16 * (j & 1)) << 16) + L::TX + t0 / 2;
        tmem_st_16x16(to, hi);
        tmem_st_16x16(to + 64, x);
      }
      if (ragged) tc::fence_async_smem();
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
        dst = a.ws + record(a, doc, row0 - seg_start, seg, head) * kRec;
        if (half == 0 && pl == 0) __stcg(dst + N * P, ex2(log_all));
      } else if (seg == segs - 1 && a.S_final != nullptr) {
        dst = a.S_final + dh * (N * P);
      }
      if (dst != nullptr) {
#pragma unroll
        for (int e = 0; e < HN; ++e) __stcg(dst + (n0 + e) * P + pl, e % 2 == 0 ? h[e / 2].x : h[e / 2].y);
      }
    }
  } else if (warp < kWarpIssue) {
    // ============================================================ ends
    set_regs<kRegsEnds<READ>>();
    if constexpr (READ) {
      const int i = 32 * q4 + lane, first = kWarpIssue - kEnds / 32;  // the group's first warp
      const int j4 = 4 * ((warp - first) >> 2);                       // this warp's 16-byte pieces of a half's rows
      const bool gated = a.z != nullptr;
      float skip[NH];
#pragma unroll
      for (int k = 0; k < NH; ++k) skip[k] = a.D != nullptr ? a.D[h0 + min(k, nh - 1)] : 0.f;
      bool ok = true;
      for (int c = 0; c < nchunks && ok; ++c) {
        const int s = c & 1, ph = (c >> 1) & 1;
#pragma unroll 1
        for (int hh = 0; hh < halves; ++hh) {
          const uint32_t zf = gated ? z_full : 0u;
          const int zp = (c * halves + hh) & 1;
          if (hh == 0) {
            ok = group(kBarEnds, kEnds, warp == first, tab_full + 8 * s, ph, x_full + 8 * s, ph, y_done, c & 1);
            if (ok && gated) ok = group(kBarEnds, kEnds, warp == first, zf, zp, 0, 0, 0, 0);
          } else {
            ok = group(kBarEnds, kEnds, warp == first, y_done + 8, c & 1, zf, zp, 0, 0);
          }
          if (!ok) break;
          tc::fence_after_sync();
          uint32_t u[2][16];
          tc::tmem_ld16(tmem + tl + L::TY + 64 * hh + 8 * j4, u[0]);
          tc::tmem_ld16(tmem + tl + L::TY + 64 * hh + 8 * j4 + 16, u[1]);
          const int k = NH == 2 ? hh : 0;
          const float sg = ex2(row_log(table(c, 0, k), i, q4)), sk = k == 0 ? skip[0] : skip[NH - 1];
          const float2 sg2 = make_float2(sg, sg), sk2 = make_float2(sk, sk);
          tc::tmem_wait_ld();
          tc::fence_before_sync();
          tc::mbar_arrive(y_free + 8 * hh);
          if (hh + 1 == halves) tc::mbar_arrive(tab_free + 8 * s);
          const auto finish = [&](auto gate) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {  // y in the place of x
              const uint32_t at = tc::sw128(i, j4 + b), xa = L::X + s * L::XT + hh * 16384 + at;
              const uint4 x4 = lds_v4(smem, xa);
              const uint32_t xw[4] = {x4.x, x4.y, x4.z, x4.w};
              float2 f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int m = 8 * b + 2 * e;
                f[e] = __ffma2_rn(sg2, make_float2(__uint_as_float(u[m / 16][m % 16]), __uint_as_float(u[m / 16][m % 16 + 1])),
                                  __fmul2_rn(sk2, widen2(xw[e])));
              }
              if constexpr (decltype(gate)::value) gate_by(lds_v4(smem, L::Z + at), f);
              *reinterpret_cast<uint4*>(smem + xa) = make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
            }
          };
          if (gated) {
            finish(std::true_type{});
            tc::mbar_arrive(z_free);
          } else {
            finish(std::false_type{});
          }
        }
        if (!ok) break;
        if (c * kC + kC > seg_n) {  // the ragged end of a document: its rows alone, through the staged tile
          tc::named_sync(kBarEnds, kEnds);
          __nv_bfloat16* const out =
              static_cast<__nv_bfloat16*>(a.out) + ((row0 + c * kC) * a.H + h0) * static_cast<long>(P);
          for (int e = tid - 32 * first; e < (seg_n - c * kC) * 8 * halves; e += kEnds) {
            const int r = e / (8 * halves), m = e % (8 * halves);
            *reinterpret_cast<uint4*>(out + static_cast<long>(r) * a.H * P + 8 * m) =
                lds_v4(smem, L::X + s * L::XT + (m >> 3) * 16384 + tc::sw128(r, m & 7));
          }
        }
        tc::fence_async_smem();
        tc::mbar_arrive(staged + 8 * s);
      }
      if (!ok) *s_abort = 1;
    }
  } else {
    set_regs<kRegsRest>();  // one call site for the whole warpgroup
    if (warp == kWarpIssue) {
      // ========================================================== MMA issue (the whole warp)
      constexpr uint32_t kIdTile = tc::idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdInc = tc::idesc_bf16(128, N, false, true);
      constexpr uint32_t kIdY = tc::idesc_bf16(128, 64, false, false), kIdMx = tc::idesc_bf16(128, 64, false, true);
      const auto all = [](bool mine) { return __all_sync(0xffffffffu, mine) != 0; };
      const uint32_t d_c = desc_low(base + L::C, 16), d_h = desc_low(base + L::H, 16);
      bool ok = true;
      for (int c = 0; c < nchunks; ++c) {
        const int s = c & 1, ph = (c >> 1) & 1;
        const uint32_t d_bk = desc_low(base + L::B + s * L::NT, 16);
        const uint32_t d_bm = desc_low(base + L::B + s * L::NT, 16384);
        ok = wait(b_full + 8 * s, ph);
        if constexpr (READ) {
          ok = all(ok && wait(c_full, c & 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 4
          for (int k = 0; k < N / 16; ++k) {
            const uint32_t ko = (k / 4) * 1024 + (k % 4) * 2;
            mma(tmem + L::TG, d_c + ko, d_bk + ko, kIdTile, k > 0);
          }
          commit(g_done);
          ok = all(wait(h_ready, c & 1));
#pragma unroll 1
          for (int hh = 0; hh < halves && ok; ++hh) {  // C h^T, 64 columns each
            ok = all(c == 0 || wait(y_free + 8 * hh, (c - 1) & 1));
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 4
            for (int k = 0; k < N / 16; ++k) {
              const uint32_t ko = (k / 4) * 1024 + (k % 4) * 2;
              mma(tmem + L::TY + 64 * hh, d_c + ko, d_h + hh * 512 + ko, kIdY, k > 0);
            }
          }
          if (!ok) break;
          commit(yoff_done);
        }
        ok = all(ok && wait(xw_ready, c & 1));
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 4
        for (int k = 0; k < 16; ++k)  // the high parts of the 128 tokens, then the low ones
          mma_ta(tmem + L::TI, tmem + L::TX + 8 * k, d_bm + (k & 7) * 128, kIdInc, k > 0);
        commit(inc_done);
        if constexpr (READ) {
          ok = all(wait(m_ready, c & 1) && wait(x_full + 8 * s, ph));
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t d_x = desc_low(base + L::X + s * L::XT, 16384);
#pragma unroll 1
          for (int hh = 0; hh < halves; ++hh) {  // M x
            const uint32_t tm = tmem + L::TG + (NH == 2 ? 8 * hh : 0);
#pragma unroll 4
            for (int k = 0; k < kC / 16; ++k)
              mma_ta(tmem + L::TY + 64 * hh, tm + 16 * k, d_x + hh * 1024 + k * 128, kIdMx, 1u);
            commit(y_done + 8 * hh);
          }
        }
      }
      if (!ok) *s_abort = 1;
      // no product is under way when TMEM and the tiles are given up
      commit(drain);
      last(drain, 0);
    } else {
      // ========================================================== TMA: one thread for B and C, for x and out, for z
      const int xc = h0 * P, nc = g * N, row = static_cast<int>(row0);
      const uint32_t xbytes = (NH == 1 ? 2 : nh) * 16384u;
      bool ok = true;
      if (warp == kWarpLoad && lane == 0) {
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
        int nb = 0, ncl = 0;  // loads issued
        if (nchunks > 0) {
          load_b(nb++);
          if (READ) load_c(ncl++);
          if (nchunks > 1) load_b(nb++);
        }
        for (int c = 0; c < nchunks; ++c) {
          if constexpr (READ) {
            ok = wait(yoff_done, c & 1);
            if (!ok) break;
            if (c + 1 < nchunks) load_c(ncl++);
          }
          ok = wait(inc_done, c & 1);
          if (!ok) break;
          if (c + 2 < nchunks) load_b(nb++);
        }
        if (!ok) *s_abort = 1;
        if (*s_abort) {  // no copy is under way when the tiles are given up: the last load of each buffer
          for (int i = 0; i < 2; ++i)
            if (nb > i) last(b_full + 8 * i, ((nb - 1 - i) >> 1) & 1);
          if (ncl > 0) last(c_full, (ncl - 1) & 1);
        }
      } else if (warp == kWarpX && lane == 0) {
        const auto load_x = [&](int c) {
          tc::mbar_arrive_expect_tx(x_full + 8 * (c & 1), xbytes);
          for (uint32_t j = 0; j < xbytes / 16384; ++j)
            tc::tma_load_3d(base + L::X + (c & 1) * L::XT + j * 16384, &maps.x, xc + 64 * j, 0, row + c * kC,
                            x_full + 8 * (c & 1));
          if (READ && a.z != nullptr)  // the gates as far as L2
            for (uint32_t j = 0; j < xbytes / 16384; ++j) tc::tma_prefetch_3d(&maps.z, xc + 64 * j, 0, row + c * kC);
        };
        int nx = 0;
        for (; nx < 2 && nx < nchunks; ++nx) load_x(nx);
        for (int c = 0; c < nchunks; ++c) {
          const int s = c & 1, ph = (c >> 1) & 1;
          // (without reading: x has been taken before the increment's products)
          ok = READ ? wait(staged + 8 * s, ph) : wait(inc_done, c & 1);
          if (!ok) break;
          if (READ && c * kC + kC <= seg_n) {  // a whole chunk was staged
            for (uint32_t j = 0; j < xbytes / 16384; ++j)
              tc::tma_store_3d(&maps.out, base + L::X + s * L::XT + j * 16384, xc + 64 * j, 0, row + c * kC);
            tc::bulk_commit();
            tc::bulk_wait_read0();  // the buffer may be refilled once the store has read it
          }
          if (c + 2 < nchunks) load_x(nx++);
        }
        if (!ok) *s_abort = 1;
        tc::bulk_wait0();
        if (*s_abort)
          for (int i = 0; i < 2; ++i)
            if (nx > i) last(x_full + 8 * i, ((nx - 1 - i) >> 1) & 1);
      } else if (READ && warp == kWarpZ && lane == 0 && a.z != nullptr) {
        int nz = 0;
        for (; nz < nchunks * halves; ++nz) {
          if (nz > 0) ok = wait(z_free, (nz - 1) & 1);
          if (!ok) break;
          tc::mbar_arrive_expect_tx(z_full, 16384);
          tc::tma_load_3d(base + L::Z, &maps.z, xc + 64 * (nz % halves), 0, row + nz / halves * kC, z_full);
        }
        if (!ok) *s_abort = 1;
        if (nz > 0 && *s_abort) last(z_full, (nz - 1) & 1);
      }
    }
  }

  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (*s_abort && tid == 0 && a.docs.dev_status != nullptr) atomicOr(a.docs.dev_status, kDevInternal);
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  if (READ) end_behind_records(a);
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
cudaError_t both(SsmArgs a, cudaStream_t stream) {
  if (a.sorted) {
    int* const order = reinterpret_cast<int*>(a.ws);
    const cudaError_t e = launch_doc_order(a.docs.cu_seqlens, a.docs.n_docs, a.docs.total_rows, order, stream);
    if (e != cudaSuccess) return e;
    a.order = order;
  }
  Maps maps;
  memset(&maps, 0, sizeof(maps));  // no rows: the kernels issue no copy
  const long rows = a.docs.total_rows, wide = static_cast<long>(a.H) * P, narrow = static_cast<long>(a.G) * N;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    e = make_map(&maps.x, a.x, rows, wide, a.xs);
    if (e == cudaSuccess) e = make_map(&maps.b, a.B, rows, narrow, a.bs);
    if (e == cudaSuccess) e = make_map(&maps.c, a.C, rows, narrow, a.cs);
    if (e == cudaSuccess && a.z != nullptr) e = make_map(&maps.z, a.z, rows, wide, a.zs);
    if (e == cudaSuccess) e = make_map(&maps.out, a.out, rows, wide, wide);
  }
  if (e == cudaSuccess && a.nseg > 1) e = go<P, N, false>(a, maps, false, stream);
  if (e == cudaSuccess && a.nseg > 1) e = launch_ssm_prefix(a, stream);
  return e != cudaSuccess ? e : go<P, N, true>(a, maps, a.nseg > 1, stream);
}

}  // namespace

bool ssm_tc_supported(DType dt, int P, int N) {
  return dt == DType::BF16 && (P == 64 || P == 128) && (N == 64 || N == 128);
}

// Segments of a document, by an estimate in units of one chunk of the scan: waves of one CTA an SM, each its chunks
// and 1.5 of set-up; kernel A's chunks cost 0.6. Of a document shorter than the longest, the CTAs without a segment
// cost 0.35 each (1.65 us: 1100 documents of 7 tokens x 16 heads of 64, N = 64, called with room for 60 segments each:
// 12.1 ms, without 0.52). A longer plan has to be 5 % faster. Packed documents whole, the longest first, take the
// longest one's time or their share of an SM, whichever is more (65536 tokens x 32 heads of 64 in documents of 128 to
// 8192: cut 373 us, whole and sorted 270). The sort compares every pair (4.7 us for 256 documents, 31 for 1024): more than
// 1024 come in their own order, and the longest may begin last.
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
    if (nseg > 1 && a.packed) cost += 2 * 0.35 / 152.0 * static_cast<double>(units * docs) * (nseg - per_doc);
    if (cost < 0.95 * best_cost) {
      best_cost = cost;
      best.nseg = static_cast<int>(nseg);
      best.seg_len = static_cast<int>(len) * kC;
    }
  }
  if (a.packed) {
    const bool sort = docs <= 1024;
    const double most = static_cast<double>(longest);
    const double each = units * (static_cast<double>(a.docs.total_rows) / kC + 0.5 * docs) / 152.0;
    if ((sort ? std::max(most, each) : most + each) + 2.5 < best_cost) {
      best.nseg = 1;
      best.seg_len = static_cast<int>(longest) * kC;
      best.sorted = sort && docs > 1;
    }
  }
  best.ws_bytes = static_cast<size_t>(ssm_records(a, best.nseg, best.seg_len)) * a.H *
                  (static_cast<size_t>(a.N) * a.P + kSsmRecTail) * 4;
  if (best.sorted) best.ws_bytes = static_cast<size_t>(docs) * sizeof(int);  // (a whole document has no records)
  return best;
}

cudaError_t launch_ssm_tc(const SsmArgs& a, cudaStream_t stream) {
  if (a.P == 64) return a.N == 64 ? both<64, 64>(a, stream) : both<64, 128>(a, stream);
  return a.N == 64 ? both<128, 64>(a, stream) : both<128, 128>(a, stream);
}

}  // namespace rapt
