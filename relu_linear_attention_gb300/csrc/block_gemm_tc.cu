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
// A pair of CTAs on two SMs forms one tile of 256 rows x up to 256 accumulator columns (cta_group::2):
// each CTA loads its 128 rows of A and its half of B, and holds its 128 rows of the accumulator; an SM
// then reads half of what two single tiles would (one CTA a tile, 128 x 256: 1480 TFLOP/s where pairs
// reach 1890 on 16384 x 2048 x 5504). Pairs are persistent; one walks its whole tiles, then its share of
// the tiles that are left over for less than a full round of all pairs: those are cut along the sum,
// evenly, and their fp32 parts go to the workspace, where a second launch adds them in order. Roles in
// a CTA:
//   warp 0     one thread streams 64-deep slices of A and B by TMA into a ring of five stages, in the
//              128-byte-swizzled layout that the tensor core reads (K-major: rows of 64 k; MN-major:
//              blocks of 64 columns, one row per k);
//   warp 1     in the pair's even CTA one thread issues the products into one of two accumulators;
//   warps 2-9  epilogue, two warps per TMEM lane quarter (half of the columns each): the other
//              accumulator is being filled meanwhile. Each warp stages 32 rows x 64 columns of bf16 in
//              one of its own two buffers and one lane stores them by TMA, which clips ragged edges: no
//              warp waits for another. GluGrad's dh comes the same way, a tile ahead.
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

constexpr int kBM = 128, kBK = 64;         // rows of a CTA, depth of a slice
constexpr int kPairRows = 2 * kBM;         // rows of a tile
constexpr int kAccCols = 256;              // TMEM columns of an accumulator: the widest tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr long long kWait = 2000000000LL;  // ~1 s of SM cycles
constexpr uint32_t kBox = 64 * 64 * 2;     // an MN-major block: 64 k x 64 columns
constexpr uint32_t kA = kBM * kBK * 2;     // a CTA's A of a slice
constexpr uint32_t kB = kA;                // a CTA's B of a slice: up to 128 columns
constexpr uint32_t kStage = kA + kB;
constexpr int kStages = 5;
constexpr uint32_t kStaged = 32 * 64 * 2;  // a staged 32 x 64 piece of a result
constexpr uint32_t kOut = kStages * kStage;
constexpr uint32_t kBar = kOut + 2 * kEpiWarps * kStaged;  // full[S], empty[S], accf[2], acce[2], dh[8]
constexpr uint32_t kMisc = kBar + (2 * kStages + 4 + kEpiWarps) * 8;  // TMEM base, abort flag
constexpr uint32_t kSmem = kMisc + 16;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kRaster = 8;  // tile rows taken together

// The tensor maps of one launch: A and B of up to two terms or products, outputs, dh.
struct Maps {
  CUtensorMap a[2];
  CUtensorMap b[2];
  CUtensorMap out[2];
  CUtensorMap dh;
};

// Pairs are numbered 0 .. workers - 1 in the plan; a GPU with fewer resident pairs takes several
// numbers each. Tile t < direct is pair (t mod workers)'s, whole. The slices of the other tiles, in
// order and `padded` for each tile (its last ones may be none), are dealt out `span` to a pair.
struct GemmArgs {
  int rows, cols;            // of an output: M and F (Glu), M and K (Dx), N and K (Dw)
  int tiles_m, tiles_n;      // output tiles of one product
  int tiles;                 // of all products
  int width;                 // output columns of a tile
  int nk[2];                 // slices of the terms of one tile's sum
  bool solid_a, solid_b;     // whether an MN-major operand's map is one of blocks
  int workers, direct, span, padded;
  float* partial;            // parts of cut sums: [2 pair + piece][CTA][column / 4][row][4] fp32
  const __nv_bfloat16* dh;
  __nv_bfloat16* out[2];
  Act act;
  uint32_t* dev_status;
};

struct Tile {
  int product, m, n;
};
// kRaster tile rows at a time, column by column: the tiles in flight share few rows of A and B.
__device__ __forceinline__ Tile tile_at(int t, int tiles_m, int tiles_n) {
  Tile r;
  const int per = tiles_m * tiles_n;
  r.product = t / per;
  t -= r.product * per;
  const int band = t / (kRaster * tiles_n);
  const int first = band * kRaster, height = min(kRaster, tiles_m - first);
  t -= first * tiles_n;
  r.m = first + t % height;
  r.n = t / height;
  return r;
}

// Walks the units of a pair: whole tiles, then pieces of cut tiles.
struct Walk {
  const GemmArgs& a;
  const int stride, nk;
  int worker, next, piece;
  long at, end;  // slices of the cut tiles
  // the unit
  int tile, k0, k1, slot;  // slot: -1 whole, else where its part goes
  __device__ __forceinline__ Walk(const GemmArgs& a_, int first, int stride_)
      : a(a_), stride(stride_), nk(a_.nk[0] + a_.nk[1]), worker(first), next(first), piece(0) {
    start();
  }
  __device__ __forceinline__ void start() {
    const long all = static_cast<long>(a.tiles - a.direct) * a.padded;
    next = worker;
    piece = 0;
    at = min(static_cast<long>(worker) * a.span, all);
    end = min(at + a.span, all);
  }
  __device__ __forceinline__ bool step() {
    for (; worker < a.workers; worker += stride, start()) {
      if (next < a.direct) {
        tile = next;
        k0 = 0;
        k1 = nk;
        slot = -1;
        next += a.workers;
        return true;
      }
      if (at < end) {
        const int of = static_cast<int>(at / a.padded);
        tile = a.direct + of;
        k0 = static_cast<int>(at - static_cast<long>(of) * a.padded);
        at = min(end, static_cast<long>(of + 1) * a.padded);
        k1 = static_cast<int>(min(static_cast<long>(nk), at - static_cast<long>(of) * a.padded));
        slot = 2 * worker + piece;
        ++piece;
        return true;
      }
    }
    return false;
  }
};

__device__ __forceinline__ void to_float16(const uint32_t (&u)[16], float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void pack16(const float (&f)[16], uint32_t (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = tc::pack_bf16x2(f[2 * i], f[2 * i + 1]);
}
// 16 bf16 into columns 16 j .. 16 j + 15 of row `lane` of a staged 32 x 64 piece.
__device__ __forceinline__ void stage16(uint32_t piece, int lane, int j, const uint32_t (&u)[8]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(piece + tc::sw128(lane, 2 * j + q)), "r"(u[4 * q]),
                 "r"(u[4 * q + 1]), "r"(u[4 * q + 2]), "r"(u[4 * q + 3])
                 : "memory");
}
// Until all but the newest `N` of this warp's stores have read their buffers.
template <int N>
__device__ __forceinline__ void stage_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
  __syncwarp();
}
// Stores the staged piece at column x, row y; TMA clips what lies past an edge of the [rows, cols] output.
__device__ __forceinline__ void stage_store(uint32_t piece, int lane, const CUtensorMap* map, int x, int y,
                                            const GemmArgs& a) {
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (x < a.cols && y < a.rows) tcp::tma_store_2d(map, piece, x, y);
    tc::bulk_commit();
  }
}
// 16 bf16 straight to columns col .. col + 15 of a row (cols is a multiple of eight).
__device__ __forceinline__ void put16(__nv_bfloat16* out, int row, int col, const uint32_t (&u)[8], const GemmArgs& a) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (row < a.rows && col + 8 * q < a.cols)
      *reinterpret_cast<uint4*>(out + static_cast<long>(row) * a.cols + col + 8 * q) =
          make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
}

template <Use USE>
__global__ void __launch_bounds__(kThreads, 1)
    block_gemm_kernel(const GemmArgs a, const __grid_constant__ Maps maps) {
  constexpr bool kGlu = USE == Use::Glu || USE == Use::GluGrad;
  constexpr bool kAMn = USE == Use::Dw, kBMn = !kGlu;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(tcp::cluster_rank());
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;
  const int half = kGlu ? a.width : a.width / 2;  // columns of B that a CTA holds

  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  const uint32_t bar_full = base + kBar, bar_empty = bar_full + 8 * kStages;
  const uint32_t bar_accf = bar_empty + 8 * kStages, bar_acce = bar_accf + 16, bar_dh = bar_acce + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kMisc + 4);
  const bool run = (base & 1023u) == 0;  // uniform; the swizzled layout needs 1 KB

  if (warp == 1 && run) tcp::tmem_alloc(tc::smem_u32(s_tmem), 2 * kAccCols);
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar_full + 8 * s, 1);
      tc::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(bar_accf + 8 * b, 1);
      tc::mbar_init(bar_acce + 8 * b, 2 * kEpiWarps);
    }
    for (int e = 0; e < kEpiWarps; ++e) tc::mbar_init(bar_dh + 8 * e, 1);
    tc::mbar_fence_init();
    *s_abort = run ? 0 : 1;
  }
  tc::fence_before_sync();
  __syncthreads();
  tcp::cluster_sync();  // the other CTA's barriers are ready, too
  tc::fence_after_sync();
  const uint32_t tmem = *s_tmem;
  tc::grid_launch_dependents();
  tc::grid_dep_wait();  // what the launch before this one in the same call wrote

  if (warp == 0) {
    if (lane == 0 && run) {  // TMA producer: this CTA's rows of A and its columns of B
      const uint32_t full0 = tcp::map_rank(bar_full, 0);
      // boxes of 64 columns hold an MN-major half, one box of `half` rows a K-major one
      const int boxes = (half + 63) / 64;
      const uint32_t bytes = 2 * (kA + (kBMn ? boxes * kBox : half * kBK * 2));
      // columns c .. of an MN-major operand: one box of the block map, or a box for every block
      const auto load_blocks = [&](const CUtensorMap* map, bool solid, int blocks, uint32_t dst, int c, int k,
                                   uint32_t bar) {
        if (solid) {
          tcp::tma_load_3d(dst, map, 0, k, c / 64, bar);
        } else {
          for (int q = 0; q < blocks; ++q) tcp::tma_load_2d(dst + q * kBox, map, c + 64 * q, k, bar);
        }
      };
      long g = 0;
      bool ok = true;
      for (Walk w(a, first, stride); ok && w.step();) {
        const Tile t = tile_at(w.tile, a.tiles_m, a.tiles_n);
        const int m0 = (t.m * 2 + rank) * kBM, n0 = t.n * a.width;
        for (int kb = w.k0; kb < w.k1; ++kb, ++g) {
          const int s = static_cast<int>(g % kStages);
          if (g >= kStages && !tc::mbar_wait(bar_empty + 8 * s, ((g / kStages) - 1) & 1, kWait)) {
            ok = false;
            break;
          }
          if (rank == 0) tc::mbar_arrive_expect_tx(bar_full + 8 * s, bytes);
          const uint32_t st = base + s * kStage, bar = full0 + 8 * s;
          const int term = kb >= a.nk[0] ? 1 : 0, k = (kb - (term ? a.nk[0] : 0)) * kBK;
          if constexpr (kAMn)
            load_blocks(&maps.a[t.product], a.solid_a, 2, st, m0, k, bar);
          else
            tcp::tma_load_2d(st, &maps.a[term], k, m0, bar);
          if constexpr (kGlu)
            tcp::tma_load_2d(st + kA, &maps.b[rank], k, n0, bar);
          else
            load_blocks(&maps.b[term], a.solid_b, boxes, st + kA, n0 + rank * half, k, bar);
        }
      }
      if (!ok) *s_abort = 1;
    }
  } else if (warp == 1) {
    if (lane == 0 && run && rank == 0) {  // issuer of the products
      const uint32_t id = tc::idesc_bf16(kPairRows, 2 * half, kAMn, kBMn);
      long g = 0;
      int i = 0;
      bool ok = true;
      for (Walk w(a, first, stride); ok && w.step(); ++i) {
        const int buf = i & 1;
        if (i >= 2 && !tc::mbar_wait(bar_acce + 8 * buf, ((i / 2) - 1) & 1, kWait)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t acc = tmem + buf * kAccCols;
        for (int kb = w.k0; kb < w.k1; ++kb, ++g) {
          const int s = static_cast<int>(g % kStages);
          if (!tc::mbar_wait(bar_full + 8 * s, (g / kStages) & 1, kWait)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t st = base + s * kStage;
          // 16 k are 32 bytes of a K-major row, 16 rows (2 KB) of an MN-major block
          const uint64_t da = tc::desc_sw128(st, kAMn ? kBox : 16, 1024);
          const uint64_t db = tc::desc_sw128(st + kA, kBMn ? kBox : 16, 1024);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tcp::mma_bf16(acc, da + (kAMn ? 128 : 2) * k, db + (kBMn ? 128 : 2) * k, id,
                             (kb > w.k0 || k > 0) ? 1u : 0u);
          tcp::mma_commit(bar_empty + 8 * s);
        }
        if (ok) tcp::mma_commit(bar_accf + 8 * buf);
      }
      if (!ok) *s_abort = 1;
    }
  } else if (run) {  // epilogue warps
    const int e = warp - 2, quarter = warp & 3, side = e >> 2;
    const uint32_t tl = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t piece[2] = {base + kOut + 2 * e * kStaged, base + kOut + (2 * e + 1) * kStaged};
    const uint32_t my_dh = bar_dh + 8 * e;
    const bool staged_dh = USE == Use::GluGrad && a.width == 128;
    // GluGrad: dh of the unit after `w` into the second buffer, which the last store has read
    const auto fetch_dh = [&](const Walk& w) {
      const Tile t = tile_at(w.tile, a.tiles_m, a.tiles_n);
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(my_dh, kStaged);
        tcp::tma_load_2d(piece[1], &maps.dh, t.n * 128 + 64 * side, (t.m * 2 + rank) * kBM + 32 * quarter, my_dh);
      }
    };
    int i = 0;
    Walk w(a, first, stride);
    bool more = w.step();
    if (staged_dh && more) fetch_dh(w);
    for (; more; ++i) {
      const int buf = i & 1;
      const Tile t = tile_at(w.tile, a.tiles_m, a.tiles_n);
      const int slot = w.slot;
      const int m0 = (t.m * 2 + rank) * kBM + 32 * quarter, row = m0 + lane;
      more = w.step();
      bool ok = tc::mbar_wait(bar_accf + 8 * buf, (i / 2) & 1, kWait);
      if (staged_dh) ok = ok && tc::mbar_wait(my_dh, i & 1, kWait);
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) *s_abort = 1;
        break;
      }
      tc::fence_after_sync();
      const uint32_t acc = tmem + buf * kAccCols + tl;
      // the accumulator has been read: the next but one tile's products may overwrite it
      const auto release = [&]() {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tcp::arrive_cluster(tcp::map_rank(bar_acce + 8 * buf, 0));
      };
      if constexpr (kGlu) {
        // this warp's columns: every other group of 64 of a full tile, of 16 of a narrow one
        const int groups = a.width / 16, step = a.width == 128 ? 1 : 2, j0 = a.width == 128 ? 4 * side : side;
        const int j1 = a.width == 128 ? j0 + 4 : groups;
        uint32_t keep[4][8];  // full tiles: du as bf16, staged once dh has been read
        if (staged_dh) stage_free<0>(lane);
        if (USE == Use::Glu && a.width == 128) stage_free<1>(lane);
        const uint32_t out = USE == Use::Glu ? piece[i & 1] : piece[0];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = j0 + q * step;
          if (j < j1) {
            const int col = t.n * a.width + 16 * j;
            uint32_t ug[16], uu[16];
            tc::tmem_ld16(acc + 16 * j, ug);
            tc::tmem_ld16(acc + a.width + 16 * j, uu);
            float d[16];
            if constexpr (USE == Use::GluGrad) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t v[4] = {0, 0, 0, 0};
                if (staged_dh)
                  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                               : "r"(piece[1] + tc::sw128(lane, 2 * q + x))
                               : "memory");
                else if (row < a.rows && col + 8 * x < a.cols)
                  *reinterpret_cast<uint4*>(v) =
                      *reinterpret_cast<const uint4*>(a.dh + static_cast<long>(row) * a.cols + col + 8 * x);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  d[8 * x + 2 * y] = __uint_as_float(v[y] << 16);
                  d[8 * x + 2 * y + 1] = __uint_as_float(v[y] & 0xffff0000u);
                }
              }
            }
            tc::tmem_wait_ld();
            float gg[16], up[16], av[16], da[16];
            to_float16(ug, gg);
            to_float16(uu, up);
            act_vec<16, USE == Use::GluGrad>(a.act, gg, av, da);
            uint32_t u[8];
            if constexpr (USE == Use::Glu) {
#pragma unroll
              for (int x = 0; x < 16; ++x) up[x] *= av[x];
            } else {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                up[x] *= d[x] * da[x];  // dg
                d[x] *= av[x];          // du
              }
              pack16(d, keep[q]);
              if (a.width != 128) put16(a.out[1], row, col, keep[q], a);
            }
            pack16(up, u);
            if (a.width == 128)
              stage16(out, lane, q, u);
            else
              put16(a.out[0], row, col, u, a);
          }
        }
        release();
        if (a.width == 128) {
          const int col = t.n * 128 + 64 * side;
          stage_store(out, lane, &maps.out[0], col, m0, a);
          if constexpr (USE == Use::GluGrad) {
#pragma unroll
            for (int q = 0; q < 4; ++q) stage16(piece[1], lane, q, keep[q]);
            stage_store(piece[1], lane, &maps.out[1], col, m0, a);
            if (more) {
              stage_free<0>(lane);
              fetch_dh(w);
            }
          }
        }
      } else if (slot < 0) {
        // groups of 64 columns in turn, at most two a warp; one fence covers both pieces (with one each,
        // the fences took a third of the epilogue's time)
        const int groups = a.width / 64;
        stage_free<0>(lane);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int c = side + 2 * q;
          if (c < groups) {
            uint32_t v[4][16];
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::tmem_ld16(acc + 64 * c + 16 * j, v[j]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float f[16];
              uint32_t u[8];
              to_float16(v[j], f);
              pack16(f, u);
              stage16(piece[q], lane, j, u);
            }
          }
        }
        release();
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int c = side + 2 * q, x = t.n * a.width + 64 * c;
            if (c < groups && x < a.cols && m0 < a.rows) tcp::tma_store_2d(&maps.out[t.product], piece[q], x, m0);
          }
          tc::bulk_commit();
        }
      } else {
        float4* p = reinterpret_cast<float4*>(a.partial) + (static_cast<long>(slot) * 2 + rank) * (kBM * kAccCols / 4);
        const int groups = a.width / 32;
#pragma unroll 1
        for (int c = side; c < groups; c += 2) {
          uint32_t v[2][16];
#pragma unroll
          for (int j = 0; j < 2; ++j) tc::tmem_ld16(acc + 32 * c + 16 * j, v[j]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              p[(8 * c + 4 * j + q) * kBM + 32 * quarter + lane] =
                  make_float4(__uint_as_float(v[j][4 * q]), __uint_as_float(v[j][4 * q + 1]),
                              __uint_as_float(v[j][4 * q + 2]), __uint_as_float(v[j][4 * q + 3]));
        }
        release();
      }
    }
    if (lane == 0) tc::bulk_wait0();  // the stores read this CTA's shared memory
  }
  tc::fence_before_sync();
  __syncthreads();
  tcp::cluster_sync();  // no CTA leaves while the other may still signal it
  if (*s_abort && tid == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, 2u);
  tc::fence_after_sync();
  if (warp == 1 && run) tcp::tmem_dealloc(tmem, 2 * kAccCols);
}

// Adds the parts of every cut tile in order and rounds once. A CTA takes 128 rows x 16 columns of a tile:
// a thread adds two quads of columns of a row (parts are stored for reading 32 rows of a quad at once),
// and the rounded rows are stored through shared memory, 32 bytes each.
struct SumArgs {
  const float4* partial;
  int rows, cols, tiles_m, tiles_n, width, direct, span, padded;
  __nv_bfloat16* out[2];
};
__global__ void __launch_bounds__(256) part_sum_kernel(const SumArgs a) {
  __shared__ uint2 rowbuf[kBM][4 + 1];
  const int cut = blockIdx.x, rank = blockIdx.z, col0 = 16 * blockIdx.y;  // which cut tile, CTA, columns
  const Tile t = tile_at(a.direct + cut, a.tiles_m, a.tiles_n);
  const long s0 = static_cast<long>(cut) * a.padded, s1 = s0 + a.padded - 1;
  const int w0 = static_cast<int>(s0 / a.span), w1 = static_cast<int>(s1 / a.span);
  const int r = threadIdx.x & (kBM - 1), q = threadIdx.x >> 7;  // row, quads q and q + 2
  const float4* p = a.partial + static_cast<long>(rank) * (kBM * kAccCols / 4) + (col0 / 4 + q) * kBM + r;
  float4 s[2] = {};
  tc::grid_dep_wait();
#pragma unroll 4
  for (int w = w0; w <= w1; ++w) {
    // the first pair's piece is its second one where its share began before this tile
    const int slot = 2 * w + (static_cast<long>(w) * a.span < s0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = p[static_cast<long>(slot) * 2 * (kBM * kAccCols / 4) + 2 * i * kBM];
      s[i].x += v.x; s[i].y += v.y; s[i].z += v.z; s[i].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    rowbuf[r][q + 2 * i] = make_uint2(tc::pack_bf16x2(s[i].x, s[i].y), tc::pack_bf16x2(s[i].z, s[i].w));
  __syncthreads();
  const int r2 = threadIdx.x >> 1, q2 = threadIdx.x & 1;
  const int row = (t.m * 2 + rank) * kBM + r2, col = t.n * a.width + col0 + 8 * q2;
  if (row >= a.rows || col >= a.cols) return;
  const uint2 lo = rowbuf[r2][2 * q2], hi = rowbuf[r2][2 * q2 + 1];
  *reinterpret_cast<uint4*>(a.out[t.product] + static_cast<long>(row) * a.cols + col) =
      make_uint4(lo.x, lo.y, hi.x, hi.y);
}

int ceil_div(long a, long b) { return static_cast<int>((a + b - 1) / b); }

// A row-major bf16 [rows, cols] matrix in boxes of box_rows x 64 columns.
cudaError_t map_2d(CUtensorMap* m, const void* p, int rows, int cols, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(cols) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
  return encode_bf16_map(m, p, 2, dims, strides, box);
}

// An MN-major operand: a row-major bf16 [rows, cols] matrix in boxes of 64 rows (the sum's index) and
// `blocks` blocks of 64 columns, block by block as the tensor core reads them. Where the columns are
// whole blocks, they are a dimension of their own and one box brings them all: TMA takes about as long
// to start a box as to copy 4 KB. Otherwise a box is one block, so that what lies past a row's end is
// zeros and not the next row.
cudaError_t map_mn(CUtensorMap* m, const void* p, int rows, int cols, int blocks, bool solid) {
  if (!solid) return map_2d(m, p, rows, cols, 64);
  const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(cols / 64)};
  const uint64_t strides[2] = {static_cast<uint64_t>(cols) * 2, 128};
  const uint32_t box[3] = {64, 64, static_cast<uint32_t>(blocks)};
  return encode_bf16_map(m, p, 3, dims, strides, box);
}

// How a launch is dealt out. The unit of cost is a 64-deep slice of a full tile (512 cycles, 0.27 us).
constexpr int kWorkers = 76;       // pairs of a GB300's 152 SMs
constexpr double kUnit = 6.0;      // slices that a tile costs beside its own: the ends of its pipeline
constexpr double kSumLaunch = 10;  // slices of the second launch of a cut plan
struct Plan {
  int width, tiles_m, tiles_n, tiles, direct, span, padded;
  double cost;
  size_t bytes;
};
// Tiles of `width` output columns (`full` at most). A slice of a narrow tile costs more than its share of
// the products: it still loads the 256 rows of A (half of a full slice's bytes), and the loads of all
// pairs together keep L2 as busy as the tensor cores (64-column tiles ran at 290 TFLOP/s).
Plan plan_width(int rows, int cols, int products, int nk, int width, int full, bool may_cut) {
  const double part = static_cast<double>(width) / full, share = std::max(part, 0.9 * (0.5 + 0.5 * part));
  Plan p{};
  p.width = width;
  p.tiles_m = ceil_div(rows, kPairRows);
  p.tiles_n = ceil_div(cols, width);
  p.tiles = p.tiles_m * p.tiles_n * products;
  p.direct = p.tiles;
  p.span = p.padded = 1;
  p.cost = static_cast<double>(ceil_div(p.tiles, kWorkers)) * (nk * share + kUnit);
  const int left = p.tiles % kWorkers;
  if (!may_cut || left == 0) return p;
  // the tiles of the last round, cut: shares of at least four slices. Where a tile takes two pairs or
  // more, all tiles are cut at the same places: pairs then read the same slices of A and B at the same
  // time, and they meet in L2. Every pair's part is written and read once, together about 6 KB in a ns.
  int span = std::max(4, ceil_div(static_cast<long>(left) * nk, kWorkers)), padded = nk;
  if (2 * left <= kWorkers) {
    span = std::max(4, ceil_div(nk, kWorkers / left));
    padded = ceil_div(nk, span) * span;
  }
  const int pairs = ceil_div(static_cast<long>(left) * padded, span);
  const double bytes = static_cast<double>(pairs + left) * kPairRows * width * 8;
  const double cost = static_cast<double>(p.tiles / kWorkers) * (nk * share + kUnit) + span * share + 2 * kUnit +
                      kSumLaunch + bytes / 6000.0 / 270.0;
  if (cost < p.cost) {
    p.direct = p.tiles - left;
    p.span = span;
    p.padded = padded;
    p.cost = cost;
    p.bytes = static_cast<size_t>(2 * pairs) * kPairRows * kAccCols * 4;
  }
  return p;
}
// The gated products: 128 columns of g and of u a tile, or fewer (a multiple of 16) where that fills the
// pairs better: M = 256, F = 5504: 43 tiles of 128, 69 of 80.
Plan plan_glu(int M, int F, int K) {
  Plan best{};
  for (int width = 128; width >= 48; width -= 16) {
    const Plan p = plan_width(M, F, 1, ceil_div(K, kBK), width, 128, false);
    if (width == 128 || p.cost < 0.95 * best.cost) best = p;
  }
  return best;
}
// The others: 256 columns, or 192, 128 or 64.
Plan plan_sum(int rows, int cols, int products, int nk) {
  Plan best{};
  for (int width = 256; width >= 64; width -= 64) {
    const Plan p = plan_width(rows, cols, products, nk, width, 256, true);
    if (width == 256 || p.cost < 0.97 * best.cost) best = p;
  }
  return best;
}
Plan plan_dx(int M, int N, int K, int terms) { return plan_sum(M, K, 1, terms * ceil_div(N, kBK)); }
Plan plan_dw(int M, int N, int K, int products) { return plan_sum(N, K, products, ceil_div(M, kBK)); }

void deal(GemmArgs* a, const Plan& p) {
  a->width = p.width;
  a->tiles_m = p.tiles_m;
  a->tiles_n = p.tiles_n;
  a->tiles = p.tiles;
  a->direct = p.direct;
  a->span = p.span;
  a->padded = p.padded;
  a->workers = kWorkers;
}

// `after`: the launch follows another one of the same call, and may be made ready before that one ends.
template <Use USE>
cudaError_t launch(const GemmArgs& a, const Maps& maps, bool after, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const auto kernel = block_gemm_kernel<USE>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> resident[64] = {};  // pairs that run at once, per device
  int pairs = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
  if (pairs == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev].store(pairs, std::memory_order_relaxed);
  }
  const int most = a.direct < a.tiles ? a.workers : std::min(a.workers, a.direct);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(pairs, most)));
  cfg.numAttrs = after ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, maps);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t sum_parts(const GemmArgs& a, cudaStream_t stream) {
  if (a.direct == a.tiles) return cudaSuccess;
  SumArgs s{};
  s.partial = reinterpret_cast<const float4*>(a.partial);
  s.rows = a.rows;
  s.cols = a.cols;
  s.tiles_m = a.tiles_m;
  s.tiles_n = a.tiles_n;
  s.width = a.width;
  s.direct = a.direct;
  s.span = a.span;
  s.padded = a.padded;
  s.out[0] = a.out[0];
  s.out[1] = a.out[1];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.tiles - a.direct, a.width / 16, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, part_sum_kernel, s);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// dx [M, K] = sum over terms of d_t [M, N] w_t [N, K].
cudaError_t run_dx(const void* const* d, const void* const* w, int terms, void* dx, int M, int N, int K,
                   float* partial, uint32_t* dev_status, bool after, cudaStream_t stream) {
  GemmArgs a{};
  a.rows = M;
  a.cols = K;
  a.nk[0] = ceil_div(N, kBK);
  a.nk[1] = terms == 2 ? a.nk[0] : 0;
  deal(&a, plan_dx(M, N, K, terms));
  a.solid_b = K % 64 == 0 && a.width % 128 == 0;
  Maps m{};
  cudaError_t e = map_2d(&m.out[0], dx, M, K, 32);
  for (int t = 0; t < terms && e == cudaSuccess; ++t) {
    e = map_2d(&m.a[t], d[t], M, N, 128);
    if (e == cudaSuccess) e = map_mn(&m.b[t], w[t], N, K, a.width / 128, a.solid_b);
  }
  if (e != cudaSuccess) return e;
  a.partial = partial;
  a.out[0] = static_cast<__nv_bfloat16*>(dx);
  a.dev_status = dev_status;
  e = launch<Use::Dx>(a, m, after, stream);
  return e != cudaSuccess ? e : sum_parts(a, stream);
}

// dw_p [N, K] = d_p^T x for one or two d_p [M, N].
cudaError_t run_dw(const void* const* d, int products, const void* x, void* const* dw, int M, int N, int K,
                   float* partial, uint32_t* dev_status, bool after, cudaStream_t stream) {
  GemmArgs a{};
  a.rows = N;
  a.cols = K;
  a.nk[0] = ceil_div(M, kBK);
  deal(&a, plan_dw(M, N, K, products));
  a.solid_a = N % 64 == 0;
  a.solid_b = K % 64 == 0 && a.width % 128 == 0;
  Maps m{};
  cudaError_t e = map_mn(&m.b[0], x, M, K, a.width / 128, a.solid_b);
  for (int t = 0; t < products && e == cudaSuccess; ++t) {
    e = map_mn(&m.a[t], d[t], M, N, 2, a.solid_a);
    if (e == cudaSuccess) e = map_2d(&m.out[t], dw[t], N, K, 32);
    a.out[t] = static_cast<__nv_bfloat16*>(dw[t]);
  }
  if (e != cudaSuccess) return e;
  a.partial = partial;
  a.dev_status = dev_status;
  e = launch<Use::Dw>(a, m, after, stream);
  return e != cudaSuccess ? e : sum_parts(a, stream);
}

template <Use USE>
cudaError_t run_glu(const GluArgs& g, const void* dh, void* out0, void* out1, cudaStream_t stream) {
  GemmArgs a{};
  a.rows = g.M;
  a.cols = g.F;
  a.nk[0] = ceil_div(g.K, kBK);
  deal(&a, plan_glu(g.M, g.F, g.K));
  a.dh = static_cast<const __nv_bfloat16*>(dh);
  a.out[0] = static_cast<__nv_bfloat16*>(out0);
  a.out[1] = static_cast<__nv_bfloat16*>(out1);
  a.act = g.act;
  a.dev_status = g.dev_status;
  Maps m{};
  cudaError_t e = map_2d(&m.a[0], g.x, g.M, g.K, 128);
  if (e == cudaSuccess) e = map_2d(&m.b[0], g.w_gate, g.F, g.K, a.width);
  if (e == cudaSuccess) e = map_2d(&m.b[1], g.w_up, g.F, g.K, a.width);
  if (e == cudaSuccess && a.width == 128) {  // narrower tiles are stored by the threads
    e = map_2d(&m.out[0], out0, g.M, g.F, 32);
    if (e == cudaSuccess && USE == Use::GluGrad) e = map_2d(&m.out[1], out1, g.M, g.F, 32);
    if (e == cudaSuccess && USE == Use::GluGrad) e = map_2d(&m.dh, dh, g.M, g.F, 32);
  }
  return e != cudaSuccess ? e : launch<USE>(a, m, false, stream);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_glu_fwd(const GluArgs& g, void* h, cudaStream_t stream) {
  if (g.M <= kGluDecodeRows) return launch_glu_decode(g, h, stream);
  return run_glu<Use::Glu>(g, nullptr, h, nullptr, stream);
}

size_t glu_bwd_ws_bytes(int M, int F, int K, bool dx, bool dw) {
  const size_t act = up256(static_cast<size_t>(M) * F * 2);
  return 2 * act + std::max(dx ? plan_dx(M, F, K, 2).bytes : 0, dw ? plan_dw(M, F, K, 2).bytes : 0);
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
    e = run_dx(d, w, 2, dx, g.M, g.F, g.K, partial, g.dev_status, true, stream);
  }
  if (e == cudaSuccess && dw_gate != nullptr) {
    void* dw[2] = {dw_gate, dw_up};
    e = run_dw(d, 2, g.x, dw, g.M, g.F, g.K, partial, g.dev_status, true, stream);
  }
  return e;
}

size_t linear_bwd_ws_bytes(int M, int N, int K, bool dx, bool dw) {
  return std::max(dx ? plan_dx(M, N, K, 1).bytes : 0, dw ? plan_dw(M, N, K, 1).bytes : 0);
}

cudaError_t launch_linear_bwd(const void* dy, const void* x, const void* w, void* dx, void* dw, int M, int N, int K,
                              void* ws, uint32_t* dev_status, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const void* d[2] = {dy, dy};
  const void* ww[2] = {w, w};
  void* o[2] = {dw, dw};
  if (dx != nullptr) e = run_dx(d, ww, 1, dx, M, N, K, static_cast<float*>(ws), dev_status, false, stream);
  if (e == cudaSuccess && dw != nullptr)
    e = run_dw(d, 1, x, o, M, N, K, static_cast<float*>(ws), dev_status, dx != nullptr, stream);
  return e;
}

}  // namespace rapt
