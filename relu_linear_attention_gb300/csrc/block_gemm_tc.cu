// The matrix products of a block's gated feed-forward and of a projection's gradients on the
// 5th-generation tensor cores (tcgen05 + TMEM), sm_103a: bf16 operands, fp32 accumulation, one
// rounding of every result to bf16. D[m, n] = sum_k A[m, k] B[n, k], four uses of one kernel:
//
//   Glu      A = x, B = the rows of w_gate and w_up: 128 columns of g = x w_gate^T and the same 128 of
//            u = x w_up^T are the two halves of one 256-column accumulator, so act(g) u is formed in
//            the epilogue from one TMEM lane and g, u never reach memory.
//   GluGrad  the same product again (g and u are cheaper to form again than to keep: 4 M F bytes), the
//            epilogue turning dh into dg = dh u act'(g) and du = dh act(g).
//   Dx       D = sum over one or two pairs (A, W): dy W, or dg w_gate + du w_up. W [n, k] is read as it
//            lies: its rows are the sum's index, so it is an MN-major operand.
//   Dw       D = dy^T x, one or two products over the tokens that share x: both operands MN-major.
//
// One persistent CTA per SM walks units of work: an output tile of 128 rows x 256 accumulator columns,
// or where the tiles are too few to fill the GPU, one part of a tile's sum (its fp32 partial goes to
// the workspace and a second launch adds the parts in order). Roles:
//   warp 0     one thread streams 64-deep slices of A and B by TMA into a ring of stages, in the
//              128-byte-swizzled layout that the tensor core reads (K-major: rows of 64 k; MN-major:
//              blocks of 64 columns, one row per k);
//   warp 1     one thread issues the products into one of two 256-column TMEM accumulators;
//   warps 2-9  epilogue, two warps per TMEM lane quarter (half of the columns each): the other
//              accumulator is being filled meanwhile. Each warp stages 32 rows x 64 columns of bf16 in
//              its own 4 KB and one lane stores them by TMA, which clips ragged edges: no warp waits
//              for another.
// Operands past an edge are read as zero by TMA. Every wait is bounded (~1 s); a CTA whose wait gives
// up sets RAPT_DEV_INTERNAL in the optional status word and stops.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "activation.cuh"
#include "kernels.h"
#include "tc_pair.cuh"
#include "tensor_map.h"

namespace rapt {
namespace {

enum class Use { Glu, GluGrad, Dx, Dw };

constexpr int kBM = 128, kBN = 256, kBK = 64;  // per CTA: accumulator rows, accumulator columns, slice depth
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr long long kWait = 2000000000LL;  // ~1 s of SM cycles
constexpr uint32_t kBox = 64 * 64 * 2;     // an MN-major block: 64 k x 64 columns
constexpr uint32_t kHalf = 128 * kBK * 2;  // 128 rows (or columns) of a slice: 16 KB
constexpr uint32_t kStageOut = 32 * 64 * 2;
constexpr int kRaster = 8;  // tile rows taken together

template <int G>
struct Cfg {
  static constexpr int kStages = G == 1 ? 4 : 6;
  static constexpr uint32_t kA = kHalf;
  static constexpr uint32_t kB = G == 1 ? 2 * kHalf : kHalf;
  static constexpr uint32_t kStage = kA + kB;
  static constexpr uint32_t kOut = kStages * kStage;
  static constexpr uint32_t kBar = kOut + kEpiWarps * kStageOut;  // full[S], empty[S], accf[2], acce[2]
  static constexpr uint32_t kMisc = kBar + (2 * kStages + 4) * 8;  // TMEM base, abort flag
  static constexpr uint32_t kSmem = kMisc + 16;
  static_assert(kSmem <= 232448, "shared memory budget");
};

// The tensor maps of one launch: A and B of up to two terms (Glu: B of w_gate, w_up), outputs.
struct Maps {
  CUtensorMap a[2];
  CUtensorMap b[2];
  CUtensorMap out[2];
};

struct GemmArgs {
  int rows, cols;        // of an output: M and F (Glu), M and K (Dx), N and K (Dw)
  int tiles_m, tiles_n;  // output tiles of one product
  int products;          // 1, or 2 (Dw of w_gate and w_up)
  int nk[2];             // slices of the terms of one tile's sum
  int parts;             // parts of a tile's sum (1: results are stored at once)
  float* partial;        // parts > 1: [unit][CTA of the pair][column / 4][row][4] fp32
  const __nv_bfloat16* dh;
  Act act;
  uint32_t* dev_status;
};

// Unit u of a launch: product, tile origin and the slices [k0, k1) of its sum.
struct Unit {
  int product, m, n, k0, k1;
};
__device__ __forceinline__ Unit unit_at(const GemmArgs& a, int u) {
  Unit r;
  const int part = u % a.parts;
  int t = u / a.parts;
  const int per = a.tiles_m * a.tiles_n;
  r.product = t / per;
  t -= r.product * per;
  // kRaster tile rows at a time, column by column: the tiles in flight share few rows of A and B
  const int band = t / (kRaster * a.tiles_n);
  const int first = band * kRaster, height = min(kRaster, a.tiles_m - first);
  t -= first * a.tiles_n;
  r.m = first + t % height;
  r.n = t / height;
  const int nk = a.nk[0] + a.nk[1];
  r.k0 = static_cast<int>(static_cast<long>(nk) * part / a.parts);
  r.k1 = static_cast<int>(static_cast<long>(nk) * (part + 1) / a.parts);
  return r;
}

// 16 accumulator columns of this thread's lane as floats.
__device__ __forceinline__ void to_float16(const uint32_t (&u)[16], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(u[i]);
}
// 16 values as bf16 into columns 16 j .. 16 j + 15 of row `lane` of a staged 32 x 64 tile.
__device__ __forceinline__ void stage16(uint32_t tile, int lane, int j, const float (&f)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t addr = tile + tc::sw128(lane, 2 * j + q);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(tc::pack_bf16x2(f[8 * q], f[8 * q + 1])),
                 "r"(tc::pack_bf16x2(f[8 * q + 2], f[8 * q + 3])), "r"(tc::pack_bf16x2(f[8 * q + 4], f[8 * q + 5])),
                 "r"(tc::pack_bf16x2(f[8 * q + 6], f[8 * q + 7]))
                 : "memory");
  }
}
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) tc::bulk_wait_read0();
  __syncwarp();
}
// Stores the staged tile at column x, row y; TMA clips what lies past an edge of the [rows, cols] output.
__device__ __forceinline__ void stage_store(uint32_t tile, int lane, const CUtensorMap* map, int x, int y,
                                            const GemmArgs& a) {
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0 && x < a.cols && y < a.rows) {
    tcp::tma_store_2d(map, tile, x, y);
    tc::bulk_commit();
  }
}

template <Use USE, int G>
__global__ void __launch_bounds__(kThreads, 1)
    block_gemm_kernel(const GemmArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<G>;
  constexpr bool kGlu = USE == Use::Glu || USE == Use::GluGrad;
  constexpr bool kAMn = USE == Use::Dw, kBMn = !kGlu;
  constexpr int kTileN = kGlu ? 128 : 256;  // output columns of a tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = G == 1 ? 0 : tcp::cluster_rank();
  const int units = a.tiles_m * a.tiles_n * a.products * a.parts;
  const int first = blockIdx.x / G, stride = gridDim.x / G;

  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  const uint32_t bar_full = base + C::kBar, bar_empty = bar_full + 8 * C::kStages;
  const uint32_t bar_accf = bar_empty + 8 * C::kStages, bar_acce = bar_accf + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  const bool misaligned = (base & 1023u) != 0;  // uniform; the swizzled layout needs 1 KB

  if (warp == 1 && !misaligned) tcp::tmem_alloc<G>(tc::smem_u32(s_tmem), 2 * kBN);
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::mbar_init(bar_full + 8 * s, 1);
      tc::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(bar_accf + 8 * b, 1);
      tc::mbar_init(bar_acce + 8 * b, G * kEpiWarps);
    }
    tc::mbar_fence_init();
    *s_abort = misaligned ? 1 : 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (G == 2) tcp::cluster_sync();  // the other CTA's barriers are ready, too
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  const bool run = !misaligned;

  if (warp == 0) {
    if (lane == 0 && run) {  // TMA producer: this CTA's rows of A and its columns of B
      const uint32_t full0 = G == 1 ? bar_full : tcp::map_rank(bar_full, 0);
      long g = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += stride) {
        const Unit w = unit_at(a, u);
        const int m0 = (w.m * G + static_cast<int>(rank)) * kBM, n0 = w.n * kTileN;
        for (int kb = w.k0; kb < w.k1; ++kb, ++g) {
          const int s = static_cast<int>(g % C::kStages);
          if (g >= C::kStages && !tcp::wait(bar_empty + 8 * s, ((g / C::kStages) - 1) & 1, kWait)) {
            ok = false;
            break;
          }
          if (rank == 0) tc::mbar_arrive_expect_tx(bar_full + 8 * s, G * C::kStage);
          const uint32_t st = base + s * C::kStage, bar = full0 + 8 * s;
          const int term = kb >= a.nk[0] ? 1 : 0, k = (kb - (term ? a.nk[0] : 0)) * kBK;
          if constexpr (kAMn) {
            const CUtensorMap* ta = &maps.a[w.product];
            tcp::tma_load_2d<G>(st, ta, m0, k, bar);
            tcp::tma_load_2d<G>(st + kBox, ta, m0 + 64, k, bar);
          } else {
            tcp::tma_load_2d<G>(st, &maps.a[term], k, m0, bar);
          }
          const uint32_t sb = st + C::kA;
          if constexpr (kGlu) {
            if constexpr (G == 1) {
              tcp::tma_load_2d<G>(sb, &maps.b[0], k, n0, bar);
              tcp::tma_load_2d<G>(sb + kHalf, &maps.b[1], k, n0, bar);
            } else {
              tcp::tma_load_2d<G>(sb, &maps.b[rank], k, n0, bar);
            }
          } else {
            const CUtensorMap* tb = &maps.b[term];
            const int nb = n0 + static_cast<int>(rank) * 128;
#pragma unroll
            for (int q = 0; q < (G == 1 ? 4 : 2); ++q) tcp::tma_load_2d<G>(sb + q * kBox, tb, nb + 64 * q, k, bar);
          }
        }
      }
      if (!ok) *s_abort = 1;
    }
  } else if (warp == 1) {
    if (lane == 0 && run && rank == 0) {  // issuer of the products
      constexpr uint32_t ID = tc::idesc_bf16(kBM * G, kBN, kAMn, kBMn);
      long g = 0;
      int i = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += stride, ++i) {
        const Unit w = unit_at(a, u);
        const int buf = i & 1;
        if (i >= 2 && !tcp::wait(bar_acce + 8 * buf, ((i / 2) - 1) & 1, kWait)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t acc = tmem + buf * kBN;
        for (int kb = w.k0; kb < w.k1; ++kb, ++g) {
          const int s = static_cast<int>(g % C::kStages);
          if (!tcp::wait(bar_full + 8 * s, (g / C::kStages) & 1, kWait)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t st = base + s * C::kStage;
          // 16 k are 32 bytes of a K-major row, 16 rows (2 KB) of an MN-major block
          const uint64_t da = tc::desc_sw128(st, kAMn ? kBox : 16, 1024);
          const uint64_t db = tc::desc_sw128(st + C::kA, kBMn ? kBox : 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tcp::mma_bf16<G>(acc, da + (kAMn ? 128 : 2) * k, db + (kBMn ? 128 : 2) * k, ID,
                             (kb > w.k0 || k > 0) ? 1u : 0u);
          tcp::mma_commit<G>(bar_empty + 8 * s);
        }
        if (ok) tcp::mma_commit<G>(bar_accf + 8 * buf);
      }
      if (!ok) *s_abort = 1;
    }
  } else if (run) {  // epilogue warps
    const int e = warp - 2, quarter = warp & 3, half = e >> 2;
    const uint32_t tl = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t tile = base + C::kOut + e * kStageOut;
    int i = 0;
    for (int u = first; u < units; u += stride, ++i) {
      const Unit w = unit_at(a, u);
      const int buf = i & 1;
      const bool ok = tcp::wait(bar_accf + 8 * buf, (i / 2) & 1, kWait);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) *s_abort = 1;
        break;
      }
      tc::fence_after_sync();
      const int m0 = (w.m * G + static_cast<int>(rank)) * kBM + 32 * quarter;
      const uint32_t acc = tmem + buf * kBN + tl;
      if constexpr (kGlu) {
        const int col0 = w.n * kTileN + 64 * half;
        [[maybe_unused]] uint32_t keep[32];  // GluGrad: du as bf16, staged after dg
        stage_free(lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t ug[16], uu[16];
          tc::tmem_ld16(acc + 64 * half + 16 * j, ug);
          tc::tmem_ld16(acc + 128 + 64 * half + 16 * j, uu);
          float d[16];
          if constexpr (USE == Use::GluGrad) {
            const int row = m0 + lane, col = col0 + 16 * j;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
              if (row < a.rows && col + 8 * q < a.cols)
                RowLoad<__nv_bfloat16, 8>::run(a.dh + static_cast<long>(row) * a.cols + col + 8 * q, v);
#pragma unroll
              for (int x = 0; x < 8; ++x) d[8 * q + x] = v[x];
            }
          }
          tc::tmem_wait_ld();
          float gg[16], up[16], av[16], da[16];
          to_float16(ug, gg);
          to_float16(uu, up);
          act_vec<16, USE == Use::GluGrad>(a.act, gg, av, da);
          if constexpr (USE == Use::Glu) {
#pragma unroll
            for (int x = 0; x < 16; ++x) up[x] *= av[x];
            stage16(tile, lane, j, up);
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              up[x] *= d[x] * da[x];  // dg
              d[x] *= av[x];          // du
            }
            stage16(tile, lane, j, up);
#pragma unroll
            for (int x = 0; x < 8; ++x) keep[8 * j + x] = tc::pack_bf16x2(d[2 * x], d[2 * x + 1]);
          }
        }
        // the accumulator has been read: the next tile's products may overwrite it
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tcp::arrive_cluster(G == 1 ? bar_acce + 8 * buf : tcp::map_rank(bar_acce + 8 * buf, 0));
        stage_store(tile, lane, &maps.out[0], col0, m0, a);
        if constexpr (USE == Use::GluGrad) {
          stage_free(lane);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tile + tc::sw128(lane, j)),
                         "r"(keep[4 * j]), "r"(keep[4 * j + 1]), "r"(keep[4 * j + 2]), "r"(keep[4 * j + 3])
                         : "memory");
          stage_store(tile, lane, &maps.out[1], col0, m0, a);
        }
      } else if (a.parts == 1) {
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int col = 128 * half + 64 * c;
          stage_free(lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t v[16];
            float f[16];
            tc::tmem_ld16(acc + col + 16 * j, v);
            tc::tmem_wait_ld();
            to_float16(v, f);
            stage16(tile, lane, j, f);
          }
          if (c == 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tcp::arrive_cluster(G == 1 ? bar_acce + 8 * buf : tcp::map_rank(bar_acce + 8 * buf, 0));
          }
          stage_store(tile, lane, &maps.out[w.product], w.n * kTileN + col, m0, a);
        }
      } else {
        float4* p = reinterpret_cast<float4*>(a.partial) + (static_cast<long>(u) * G + rank) * (kBM * kBN / 4);
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          const int col = 128 * half + 16 * j;
          uint32_t v[16];
          tc::tmem_ld16(acc + col, v);
          tc::tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            p[(col / 4 + q) * kBM + 32 * quarter + lane] =
                make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                            __uint_as_float(v[4 * q + 3]));
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tcp::arrive_cluster(G == 1 ? bar_acce + 8 * buf : tcp::map_rank(bar_acce + 8 * buf, 0));
      }
    }
    if (lane == 0) tc::bulk_wait0();  // the stores read this CTA's shared memory
  }
  tc::fence_before_sync();
  __syncthreads();
  if constexpr (G == 2) tcp::cluster_sync();  // no CTA leaves while the other may still signal it
  if (*s_abort && tid == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, 2u);
  tc::fence_after_sync();
  if (warp == 1 && !misaligned) tcp::tmem_dealloc<G>(tmem, 2 * kBN);
}

// Adds the parts of every tile's sum in order and rounds once. One thread: one row, 16 columns.
struct SumArgs {
  const float4* partial;
  int rows, cols, tiles_m, tiles_n, parts;
  __nv_bfloat16* out[2];
};
template <int G>
__global__ void __launch_bounds__(256) part_sum_kernel(const SumArgs a) {
  const int t = blockIdx.x;  // tile of a product, in unit order
  const int seg = blockIdx.y * 2 + (threadIdx.x >> 7), r = threadIdx.x & 127;  // 16 columns, row of the CTA's 128
  GemmArgs g{};
  g.tiles_m = a.tiles_m;
  g.tiles_n = a.tiles_n;
  g.parts = 1;
  const Unit w = unit_at(g, t);
#pragma unroll
  for (int rank = 0; rank < G; ++rank) {
    const int row = (w.m * G + rank) * kBM + r, col = w.n * kBN + 16 * seg;
    if (row >= a.rows || col >= a.cols) continue;
    float4 s[4] = {};
    for (int p = 0; p < a.parts; ++p) {
      const float4* src = a.partial + ((static_cast<long>(t) * a.parts + p) * G + rank) * (kBM * kBN / 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = src[(4 * seg + q) * kBM + r];
        s[q].x += v.x; s[q].y += v.y; s[q].z += v.z; s[q].w += v.w;
      }
    }
    uint4* o = reinterpret_cast<uint4*>(a.out[w.product] + static_cast<long>(row) * a.cols + col);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (col + 8 * q >= a.cols) break;
      o[q] = make_uint4(tc::pack_bf16x2(s[2 * q].x, s[2 * q].y), tc::pack_bf16x2(s[2 * q].z, s[2 * q].w),
                        tc::pack_bf16x2(s[2 * q + 1].x, s[2 * q + 1].y),
                        tc::pack_bf16x2(s[2 * q + 1].z, s[2 * q + 1].w));
    }
  }
}

int ceil_div(long a, long b) { return static_cast<int>((a + b - 1) / b); }

// A row-major bf16 [rows, cols] matrix in boxes of box_rows x 64 columns.
cudaError_t map_2d(CUtensorMap* m, const void* p, int rows, int cols, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
  return encode_bf16_map(m, p, 2, dims, strides, box);
}

// Parts of a tile's sum: what finishes first by a count of slices per SM (or pair), where a unit
// costs kUnit slices beside its own and the second launch moves 8 bytes per partial value.
constexpr int kPlanSms = 152;
template <int G>
int plan_parts(long tiles, int nk) {
  constexpr double kUnit = 6.0, kLaunch = 14.0;
  const int workers = kPlanSms / G;
  double best = 0;
  int parts = 1;
  for (int p = 1; p <= 16 && p <= nk; ++p) {
    double cost = static_cast<double>(ceil_div(tiles * p, workers)) * (ceil_div(nk, p) + kUnit);
    // a slice is 512 cycles (0.27 us); all SMs together move about 6 KB of partials in a ns
    if (p > 1) cost += kLaunch + static_cast<double>(tiles) * p * G * kBM * kBN * 8 / 6000.0 / 270.0;
    if (p == 1 || cost < 0.97 * best) {
      best = cost;
      parts = p;
    }
  }
  return parts;
}

template <Use USE, int G>
cudaError_t launch(GemmArgs a, const Maps& maps, cudaStream_t stream) {
  using C = Cfg<G>;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const auto kernel = block_gemm_kernel<USE, G>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / G * G));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = G;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> resident[64] = {};  // CTAs or pairs that run at once, per device
  int workers = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (workers == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&workers, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (workers < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev].store(workers, std::memory_order_relaxed);
  }
  const long units = static_cast<long>(a.tiles_m) * a.tiles_n * a.products * a.parts;
  workers = static_cast<int>(std::min<long>(units, workers));
  cfg.gridDim = dim3(static_cast<unsigned>(workers * G));
  e = cudaLaunchKernelEx(&cfg, kernel, a, maps);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int G>
cudaError_t sum_parts(const GemmArgs& a, void* out0, void* out1, cudaStream_t stream) {
  SumArgs s{};
  s.partial = reinterpret_cast<const float4*>(a.partial);
  s.rows = a.rows;
  s.cols = a.cols;
  s.tiles_m = a.tiles_m;
  s.tiles_n = a.tiles_n;
  s.parts = a.parts;
  s.out[0] = static_cast<__nv_bfloat16*>(out0);
  s.out[1] = static_cast<__nv_bfloat16*>(out1);
  part_sum_kernel<G><<<dim3(a.tiles_m * a.tiles_n * a.products, kBN / 32), 256, 0, stream>>>(s);
  note_launches(1);
  return cudaGetLastError();
}

constexpr int kG = 2;

size_t partial_bytes(long tiles, int nk) {
  const int parts = plan_parts<kG>(tiles, nk);
  return parts == 1 ? 0 : static_cast<size_t>(tiles) * parts * kG * kBM * kBN * 4;
}

// dx [M, K] = sum over terms of d_t [M, N] w_t [N, K].
cudaError_t run_dx(const void* const* d, const void* const* w, int terms, void* dx, int M, int N, int K,
                   float* partial, uint32_t* dev_status, cudaStream_t stream) {
  Maps m{};
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < 2 && e == cudaSuccess; ++t) {
    e = map_2d(&m.a[t], d[t < terms ? t : 0], M, N, 128);
    if (e == cudaSuccess) e = map_2d(&m.b[t], w[t < terms ? t : 0], N, K, 64);
    if (e == cudaSuccess) e = map_2d(&m.out[t], dx, M, K, 32);
  }
  if (e != cudaSuccess) return e;
  GemmArgs a{};
  a.rows = M;
  a.cols = K;
  a.tiles_m = ceil_div(M, kBM * kG);
  a.tiles_n = ceil_div(K, kBN);
  a.products = 1;
  a.nk[0] = ceil_div(N, kBK);
  a.nk[1] = terms == 2 ? a.nk[0] : 0;
  a.parts = plan_parts<kG>(static_cast<long>(a.tiles_m) * a.tiles_n, a.nk[0] + a.nk[1]);
  a.partial = partial;
  a.dev_status = dev_status;
  e = launch<Use::Dx, kG>(a, m, stream);
  if (e != cudaSuccess || a.parts == 1) return e;
  return sum_parts<kG>(a, dx, nullptr, stream);
}

// dw_p [N, K] = d_p^T x for one or two d_p [M, N].
cudaError_t run_dw(const void* const* d, int products, const void* x, void* const* dw, int M, int N, int K,
                   float* partial, uint32_t* dev_status, cudaStream_t stream) {
  Maps m{};
  cudaError_t e = cudaSuccess;
  for (int t = 0; t < 2 && e == cudaSuccess; ++t) {
    const int p = t < products ? t : 0;
    e = map_2d(&m.a[t], d[p], M, N, 64);
    if (e == cudaSuccess) e = map_2d(&m.b[t], x, M, K, 64);
    if (e == cudaSuccess) e = map_2d(&m.out[t], dw[p], N, K, 32);
  }
  if (e != cudaSuccess) return e;
  GemmArgs a{};
  a.rows = N;
  a.cols = K;
  a.tiles_m = ceil_div(N, kBM * kG);
  a.tiles_n = ceil_div(K, kBN);
  a.products = products;
  a.nk[0] = ceil_div(M, kBK);
  a.parts = plan_parts<kG>(static_cast<long>(a.tiles_m) * a.tiles_n * products, a.nk[0]);
  a.partial = partial;
  a.dev_status = dev_status;
  e = launch<Use::Dw, kG>(a, m, stream);
  if (e != cudaSuccess || a.parts == 1) return e;
  return sum_parts<kG>(a, dw[0], products == 2 ? dw[1] : nullptr, stream);
}

template <Use USE>
cudaError_t run_glu(const GluArgs& g, const void* dh, void* out0, void* out1, cudaStream_t stream) {
  Maps m{};
  cudaError_t e = map_2d(&m.a[0], g.x, g.M, g.K, 128);
  m.a[1] = m.a[0];
  if (e == cudaSuccess) e = map_2d(&m.b[0], g.w_gate, g.F, g.K, 128);
  if (e == cudaSuccess) e = map_2d(&m.b[1], g.w_up, g.F, g.K, 128);
  if (e == cudaSuccess) e = map_2d(&m.out[0], out0, g.M, g.F, 32);
  if (e == cudaSuccess) e = map_2d(&m.out[1], out1, g.M, g.F, 32);
  if (e != cudaSuccess) return e;
  GemmArgs a{};
  a.rows = g.M;
  a.cols = g.F;
  a.tiles_m = ceil_div(g.M, kBM * kG);
  a.tiles_n = ceil_div(g.F, 128);
  a.products = 1;
  a.nk[0] = ceil_div(g.K, kBK);
  a.parts = 1;
  a.dh = static_cast<const __nv_bfloat16*>(dh);
  a.act = g.act;
  a.dev_status = g.dev_status;
  return launch<USE, kG>(a, m, stream);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t dx_bytes(int M, int N, int K, int terms) {
  return partial_bytes(static_cast<long>(ceil_div(M, kBM * kG)) * ceil_div(K, kBN), terms * ceil_div(N, kBK));
}
size_t dw_bytes(int M, int N, int K, int products) {
  return partial_bytes(static_cast<long>(ceil_div(N, kBM * kG)) * ceil_div(K, kBN) * products, ceil_div(M, kBK));
}

}  // namespace

cudaError_t launch_glu_fwd(const GluArgs& g, void* h, cudaStream_t stream) {
  if (g.M <= kGluDecodeRows) return launch_glu_decode(g, h, stream);
  return run_glu<Use::Glu>(g, nullptr, h, h, stream);
}

size_t glu_bwd_ws_bytes(int M, int F, int K, bool dx, bool dw) {
  const size_t act = up256(static_cast<size_t>(M) * F * 2);
  return 2 * act + std::max(dx ? dx_bytes(M, F, K, 2) : 0, dw ? dw_bytes(M, F, K, 2) : 0);
}

cudaError_t launch_glu_bwd(const GluArgs& g, const void* dh, void* dx, void* dw_gate, void* dw_up, void* ws,
                           cudaStream_t stream) {
  const size_t act = up256(static_cast<size_t>(g.M) * g.F * 2);
  void* dg = ws;
  void* du = static_cast<uint8_t*>(ws) + act;
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * act);
  cudaError_t e = run_glu<Use::GluGrad>(g, dh, dg, du, stream);
  const void* d[2] = {dg, du};
  if (e == cudaSuccess && dx != nullptr) {
    const void* w[2] = {g.w_gate, g.w_up};
    e = run_dx(d, w, 2, dx, g.M, g.F, g.K, partial, g.dev_status, stream);
  }
  if (e == cudaSuccess && dw_gate != nullptr) {
    void* dw[2] = {dw_gate, dw_up};
    e = run_dw(d, 2, g.x, dw, g.M, g.F, g.K, partial, g.dev_status, stream);
  }
  return e;
}

size_t linear_bwd_ws_bytes(int M, int N, int K, bool dx, bool dw) {
  return std::max(dx ? dx_bytes(M, N, K, 1) : 0, dw ? dw_bytes(M, N, K, 1) : 0);
}

cudaError_t launch_linear_bwd(const void* dy, const void* x, const void* w, void* dx, void* dw, int M, int N, int K,
                              void* ws, uint32_t* dev_status, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const void* d[2] = {dy, dy};
  const void* ww[2] = {w, w};
  void* o[2] = {dw, dw};
  if (dx != nullptr) e = run_dx(d, ww, 1, dx, M, N, K, static_cast<float*>(ws), dev_status, stream);
  if (e == cudaSuccess && dw != nullptr)
    e = run_dw(d, 1, x, o, M, N, K, static_cast<float*>(ws), dev_status, stream);
  return e;
}

}  // namespace rapt
