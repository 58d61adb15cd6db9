// The matrix products of a block's gated feed-forward and of a projection's gradients on the
// 5th-generation tensor cores (tcgen05 + TMEM), sm_103a: bf16 operands, fp32 accumulation, one
// rounding of every result to bf16. D[m, n] = sum_k A[m, k] B[n, k], in four forms:
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
// Dx and Dw are the two problems of one launch: its pairs go from the one to the other without a
// pause (2048 x 6144 x 2048: 92 us as two launches, 85 as one).
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
//              warp waits for another. GluGrad's dh comes the same way, a tile ahead, into the other.
// Operands past an edge are read as zero by TMA. Every wait is bounded (~1 s); a CTA whose wait gives
// up sets RAPT_DEV_INTERNAL in the optional status word and stops.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "kernels.h"
#include "tc_pair.cuh"
#include "tensor_map.h"

namespace rapt {
namespace {

enum class Use { Glu, GluGrad, Grads };  // Grads: problem 0 is Dx, problem 1 Dw

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

// The tensor maps of one launch: A and B of up to two terms or products of each problem (the MN-major ones
// also block by block), outputs, dh.
struct Maps {
  CUtensorMap a[2][2], a_blocks[2];
  CUtensorMap b[2][2], b_blocks[2][2];
  CUtensorMap out[2][2];
  CUtensorMap dh;
};

// One matrix product, or two of the same shape. Pairs are numbered 0 .. workers - 1 in the plan; a GPU
// with fewer resident pairs takes several numbers each. Tile t < direct is pair (t mod workers)'s, whole.
// The slices of the other tiles, in order and `padded` for each tile (its last ones may be none), are
// dealt out `span` to a pair. The second problem's pairs are numbered from pair `turn`, where the
// first's last round ended.
struct Problem {
  int rows, cols;        // of an output: M and F (Glu), M and K (Dx), N and K (Dw)
  int tiles_m, tiles_n;  // output tiles of one product
  int tiles;             // of all products
  int width;             // output columns of a tile
  int nk0, nk;           // slices of a tile's sum: of its first term, in all
  int direct, span, padded, turn;
  int slot0;             // first of its parts' places in the workspace
  int solid_a, solid_b;  // columns of the MN-major A (Dw) and B that their block maps have
  __nv_bfloat16* out[2];
  int pitch;  // elements of an output's row (Glu)
};
struct GemmArgs {
  Problem p[2];
  int workers;
  float* partial;  // parts of cut sums: [slot0 + 2 pair + piece][CTA][column / 4][row][4] fp32
  const __nv_bfloat16* dh;
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

// Walks the units of a pair: of each problem its whole tiles, then its pieces of cut tiles.
struct Walk {
  const GemmArgs& a;
  const int stride;
  int worker, q, next, piece, number;
  long at, end;  // slices of the cut tiles
  // the unit
  int tile, k0, k1, slot;  // slot: -1 whole, else where its part goes
  __device__ __forceinline__ Walk(const GemmArgs& a_, int first, int stride_) : a(a_), stride(stride_), worker(first), q(0) {
    open();
  }
  __device__ __forceinline__ const Problem& problem() const { return a.p[q]; }
  __device__ __forceinline__ void open() {
    const Problem& p = a.p[q];
    number = worker - p.turn + (worker < p.turn ? a.workers : 0);
    const long all = static_cast<long>(p.tiles - p.direct) * p.padded;
    next = number;
    piece = 0;
    at = min(static_cast<long>(number) * p.span, all);
    end = min(at + p.span, all);
  }
  __device__ __forceinline__ bool step() {
    while (worker < a.workers) {
      const Problem& p = a.p[q];
      if (next < p.direct) {
        tile = next;
        k0 = 0;
        k1 = p.nk;
        slot = -1;
        next += a.workers;
        return true;
      }
      if (at < end) {
        const int of = static_cast<int>(at / p.padded);
        tile = p.direct + of;
        k0 = static_cast<int>(at - static_cast<long>(of) * p.padded);
        at = min(end, static_cast<long>(of + 1) * p.padded);
        k1 = static_cast<int>(min(static_cast<long>(p.nk), at - static_cast<long>(of) * p.padded));
        slot = p.slot0 + 2 * number + piece;
        ++piece;
        return true;
      }
      if (q == 0) {
        q = 1;
      } else {
        q = 0;
        worker += stride;
        if (worker >= a.workers) return false;
      }
      open();
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
                                            const Problem& p) {
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (x < p.cols && y < p.rows) tcp::tma_store_2d(map, piece, x, y);
    tc::bulk_commit();
  }
}
// 16 bf16 straight to columns col .. col + 15 of a row (cols is a multiple of eight).
__device__ __forceinline__ void put16(__nv_bfloat16* out, int row, int col, const uint32_t (&u)[8], const Problem& p) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (row < p.rows && col + 8 * q < p.cols)
      *reinterpret_cast<uint4*>(out + static_cast<long>(row) * p.pitch + col + 8 * q) =
          make_uint4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
}

template <Use USE>
__global__ void __launch_bounds__(kThreads, 1)
    block_gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ Maps maps) {
  constexpr bool kGlu = USE == Use::Glu || USE == Use::GluGrad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(tcp::cluster_rank());
  const int first = blockIdx.x / 2, stride = gridDim.x / 2;

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

  tcp::Ring<kStages> ring;  // of the thread that loads, of the one that multiplies
  if (warp == 0) {
    if (lane == 0 && run) {  // TMA producer: this CTA's rows of A and its columns of B
      const uint32_t full0 = tcp::map_rank(bar_full, 0);
      bool ok = true;
      // one slice after another into the ring: load(stage, full barrier, slice) issues its copies
      const auto stream = [&](int k0, int k1, uint32_t bytes, const auto& load) {
        for (int kb = k0; kb < k1; ++kb, ring.step()) {
          if (ring.round > 0 && !tcp::wait(bar_empty + 8 * ring.s, (ring.round - 1) & 1, kWait)) {
            ok = false;
            return;
          }
          if (rank == 0) tc::mbar_arrive_expect_tx(bar_full + 8 * ring.s, bytes);
          load(base + ring.s * kStage, full0 + 8 * ring.s, kb);
        }
      };
      for (Walk w(a, first, stride); ok && w.step();) {
        const Problem& p = w.problem();
        const Tile t = tile_at(w.tile, p.tiles_m, p.tiles_n);
        const int m0 = (t.m * 2 + rank) * kBM, n0 = t.n * p.width;
        if constexpr (kGlu) {
          const CUtensorMap* mb = &maps.b[0][rank];
          stream(w.k0, w.k1, 2 * (kA + p.width * kBK * 2), [&](uint32_t st, uint32_t bar, int kb) {
            tcp::tma_load_2d(st, &maps.a[0][0], kb * kBK, m0, bar);
            tcp::tma_load_2d(st + kA, mb, kb * kBK, n0, bar);
          });
        } else {
          const int half = p.width / 2, blocks = half / 64, nb = n0 + rank * half;
          const uint32_t bytes = 2 * (kA + blocks * kBox);
          const bool solid_a = m0 + kBM <= p.solid_a, solid_b = nb + half <= p.solid_b;
          // columns c .. of an MN-major operand: one box of the block map where it has them all, or a box
          // for every block
          const auto load_mn = [&](const CUtensorMap* map, const CUtensorMap* by_block, bool solid, int n, uint32_t dst,
                                   int c, int k, uint32_t bar) {
            if (solid) {
              tcp::tma_load_3d(dst, by_block, 0, k, c / 64, bar);
            } else {
              tcp::tma_load_2d(dst, map, c, k, bar);
              if (n > 1) tcp::tma_load_2d(dst + kBox, map, c + 64, k, bar);
            }
          };
          if (w.q == 0) {
            const int nk0 = p.nk0;
            for (int term = 0; term < 2 && ok; ++term) {
              const CUtensorMap *ma = &maps.a[0][term], *mb = &maps.b[0][term], *bb = &maps.b_blocks[0][term];
              const int skip = term * nk0;  // slices of the terms before
              stream(max(w.k0, skip), min(w.k1, skip + nk0), bytes, [&](uint32_t st, uint32_t bar, int kb) {
                const int k = (kb - skip) * kBK;
                tcp::tma_load_2d(st, ma, k, m0, bar);
                load_mn(mb, bb, solid_b, blocks, st + kA, nb, k, bar);
              });
            }
          } else {
            const CUtensorMap *ma = &maps.a[1][t.product], *mb = &maps.b[1][0];
            const CUtensorMap *ab = &maps.a_blocks[t.product], *bb = &maps.b_blocks[1][0];
            stream(w.k0, w.k1, bytes, [&](uint32_t st, uint32_t bar, int kb) {
              load_mn(ma, ab, solid_a, 2, st, m0, kb * kBK, bar);
              load_mn(mb, bb, solid_b, blocks, st + kA, nb, kb * kBK, bar);
            });
          }
        }
      }
      if (!ok) *s_abort = 1;
    }
  } else if (warp == 1) {
    if (lane == 0 && run && rank == 0) {  // issuer of the products
      tcp::Ring<2> accs;
      bool ok = true;
      // the slices of one unit; A_MN: A is MN-major (Dw)
      const auto multiply = [&](int slices, uint32_t acc, uint32_t id, auto a_mn) {
        constexpr bool kAMn = decltype(a_mn)::value, kBMn = !kGlu;
        // 16 k are 32 bytes of a K-major row, 16 rows (2 KB) of an MN-major block
        constexpr int kStepA = kAMn ? 128 : 2, kStepB = kBMn ? 128 : 2;
        const uint64_t da0 = tc::desc_sw128(base, kAMn ? kBox : 16, 1024);
        const uint64_t db0 = tc::desc_sw128(base + kA, kBMn ? kBox : 16, 1024);
        for (int q = 0; q < slices; ++q, ring.step()) {
          if (!tcp::wait(bar_full + 8 * ring.s, ring.round & 1, kWait)) {
            ok = false;
            return;
          }
          tc::fence_after_sync();
          const uint64_t da = da0 + ring.s * (kStage / 16), db = db0 + ring.s * (kStage / 16);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tcp::mma_bf16(acc, da + kStepA * k, db + kStepB * k, id, (q > 0 || k > 0) ? 1u : 0u);
          tcp::mma_commit(bar_empty + 8 * ring.s);
        }
      };
      for (Walk w(a, first, stride); ok && w.step(); accs.step()) {
        const int width = w.problem().width;
        const bool a_mn = !kGlu && w.q == 1;
        const uint32_t id = tc::idesc_bf16(kPairRows, kGlu ? 2 * width : width, a_mn, !kGlu);
        if (accs.round > 0 && !tcp::wait(bar_acce + 8 * accs.s, (accs.round - 1) & 1, kWait)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t acc = tmem + accs.s * kAccCols;
        if (a_mn)
          multiply(w.k1 - w.k0, acc, id, std::true_type{});
        else
          multiply(w.k1 - w.k0, acc, id, std::false_type{});
        if (ok) tcp::mma_commit(bar_accf + 8 * accs.s);
      }
      if (!ok) *s_abort = 1;
    }
  } else if (run) {  // epilogue warps
    const int e = warp - 2, quarter = warp & 3, side = e >> 2;
    const uint32_t tl = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t piece[2] = {base + kOut + 2 * e * kStaged, base + kOut + (2 * e + 1) * kStaged};
    const uint32_t my_dh = bar_dh + 8 * e;
    const bool staged_dh = USE == Use::GluGrad && a.p[0].width == 128;
    // GluGrad: dh of unit `w` into the second buffer
    const auto fetch_dh = [&](const Walk& w) {
      const Tile t = tile_at(w.tile, a.p[0].tiles_m, a.p[0].tiles_n);
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
      const Problem& p = w.problem();
      const Tile t = tile_at(w.tile, p.tiles_m, p.tiles_n);
      const int slot = w.slot;
      [[maybe_unused]] const CUtensorMap* outs = maps.out[w.q];
      const int m0 = (t.m * 2 + rank) * kBM + 32 * quarter, row = m0 + lane;
      more = w.step();
      bool ok = tcp::wait(bar_accf + 8 * buf, (i / 2) & 1, kWait);
      if (staged_dh) ok = tcp::wait(my_dh, i & 1, kWait) && ok;  // in any case: no copy is left under way
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
        const int groups = p.width / 16, step = p.width == 128 ? 1 : 2, j0 = p.width == 128 ? 4 * side : side;
        const int j1 = p.width == 128 ? j0 + 4 : groups;
        // full tiles: this unit's dh to registers, so that the next one's is under way during the arithmetic
        // (fetched after it, 16384 x 128 x 4096 with dx: 172 us, 154 so); du as bf16, staged where dg was
        [[maybe_unused]] uint32_t dh[4][8], keep[4][8];
        if (staged_dh) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(dh[q / 2][4 * (q % 2)]), "=r"(dh[q / 2][4 * (q % 2) + 1]),
                           "=r"(dh[q / 2][4 * (q % 2) + 2]), "=r"(dh[q / 2][4 * (q % 2) + 3])
                         : "r"(piece[1] + tc::sw128(lane, q))
                         : "memory");
          __syncwarp();
          if (more) fetch_dh(w);
          stage_free<0>(lane);
        }
        if (USE == Use::Glu && p.width == 128) stage_free<1>(lane);
        const uint32_t out = USE == Use::Glu ? piece[i & 1] : piece[0];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = j0 + q * step;
          if (j < j1) {
            const int col = t.n * p.width + 16 * j;
            uint32_t ug[16], uu[16];
            tc::tmem_ld16(acc + 16 * j, ug);
            tc::tmem_ld16(acc + p.width + 16 * j, uu);
            float d[16];
            if constexpr (USE == Use::GluGrad) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t v[4] = {0, 0, 0, 0};
                if (staged_dh) {
#pragma unroll
                  for (int y = 0; y < 4; ++y) v[y] = dh[q][4 * x + y];
                } else if (row < p.rows && col + 8 * x < p.cols)
                  *reinterpret_cast<uint4*>(v) =
                      *reinterpret_cast<const uint4*>(a.dh + static_cast<long>(row) * p.cols + col + 8 * x);
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
              if (p.width != 128) put16(p.out[1], row, col, keep[q], p);
            }
            pack16(up, u);
            if (p.width == 128)
              stage16(out, lane, q, u);
            else
              put16(p.out[0], row, col, u, p);
          }
        }
        release();
        if (p.width == 128) {
          const int col = t.n * 128 + 64 * side;
          stage_store(out, lane, &outs[0], col, m0, p);
          if constexpr (USE == Use::GluGrad) {
            stage_free<0>(lane);
#pragma unroll
            for (int q = 0; q < 4; ++q) stage16(out, lane, q, keep[q]);
            stage_store(out, lane, &outs[1], col, m0, p);
          }
        }
      } else if (slot < 0) {
        // groups of 64 columns in turn, at most two a warp; one fence covers both pieces (with one each,
        // the fences took a third of the epilogue's time)
        const int groups = p.width / 64;
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
            const int c = side + 2 * q, x = t.n * p.width + 64 * c;
            if (c < groups && x < p.cols && m0 < p.rows) tcp::tma_store_2d(&outs[t.product], piece[q], x, m0);
          }
          tc::bulk_commit();
        }
      } else {
        float4* part = reinterpret_cast<float4*>(a.partial) + (static_cast<long>(slot) * 2 + rank) * (kBM * kAccCols / 4);
        const int groups = p.width / 32;
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
              part[(8 * c + 4 * j + q) * kBM + 32 * quarter + lane] =
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
  if (tid == 0 && run && *s_abort) {  // given up: what is on its way to either CTA still lands
    for (int s = 0; s < (rank == 0 ? kStages : 0); ++s) {
      const uint32_t rounds = ring.round + (s < ring.s ? 1 : 0);
      if (rounds > 0) tcp::wait(bar_full + 8 * s, (rounds - 1) & 1, kWait);
    }
    // half a millisecond for what no phase here stands for: slices that the other CTA fetched further on, and
    // products of an issuer that went on without the epilogue
    for (const long long t0 = clock64(); clock64() - t0 < (1 << 20);) __nanosleep(1000);
  }
  __syncwarp();
  tcp::cluster_sync();  // no CTA leaves while the other may still signal it
  if (*s_abort && tid == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, 2u);
  tc::fence_after_sync();
  if (warp == 1 && run) tcp::tmem_dealloc(tmem, 2 * kAccCols);
}

// Adds the parts of every cut tile in order and rounds once. A CTA takes 128 rows x 16 columns of a tile:
// a thread adds two quads of columns of a row (parts are stored for reading 32 rows of a quad at once),
// and the rounded rows are stored through shared memory, 32 bytes each.
__global__ void __launch_bounds__(256) part_sum_kernel(const __grid_constant__ GemmArgs a, int cut0) {
  __shared__ uint2 rowbuf[kBM][4 + 1];
  const int q_ = static_cast<int>(blockIdx.x) >= cut0 ? 1 : 0;  // problem
  const Problem& p = a.p[q_];
  const int cut = blockIdx.x - (q_ ? cut0 : 0), rank = blockIdx.z, col0 = 16 * blockIdx.y;  // tile, CTA, columns
  if (col0 >= p.width) return;
  const Tile t = tile_at(p.direct + cut, p.tiles_m, p.tiles_n);
  const long s0 = static_cast<long>(cut) * p.padded, s1 = s0 + p.padded - 1;
  const int w0 = static_cast<int>(s0 / p.span), w1 = static_cast<int>(s1 / p.span);
  const int r = threadIdx.x & (kBM - 1), q = threadIdx.x >> 7;  // row, quads q and q + 2
  const float4* from = reinterpret_cast<const float4*>(a.partial) +
                       (static_cast<long>(p.slot0) * 2 + rank) * (kBM * kAccCols / 4) + (col0 / 4 + q) * kBM + r;
  float4 s[2] = {};
  tc::grid_dep_wait();
#pragma unroll 4
  for (int w = w0; w <= w1; ++w) {
    // the first pair's piece is its second one where its share began before this tile
    const int slot = 2 * w + (static_cast<long>(w) * p.span < s0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = from[static_cast<long>(slot) * 2 * (kBM * kAccCols / 4) + 2 * i * kBM];
      s[i].x += v.x; s[i].y += v.y; s[i].z += v.z; s[i].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    rowbuf[r][q + 2 * i] = make_uint2(tc::pack_bf16x2(s[i].x, s[i].y), tc::pack_bf16x2(s[i].z, s[i].w));
  __syncthreads();
  const int r2 = threadIdx.x >> 1, q2 = threadIdx.x & 1;
  const int row = (t.m * 2 + rank) * kBM + r2, col = t.n * p.width + col0 + 8 * q2;
  if (row >= p.rows || col >= p.cols) return;
  const uint2 lo = rowbuf[r2][2 * q2], hi = rowbuf[r2][2 * q2 + 1];
  *reinterpret_cast<uint4*>((t.product ? p.out[1] : p.out[0]) + static_cast<long>(row) * p.cols + col) =
      make_uint4(lo.x, lo.y, hi.x, hi.y);
}

int ceil_div(long a, long b) { return static_cast<int>((a + b - 1) / b); }

// A row-major bf16 [rows, cols] matrix, `pitch` elements a row, in boxes of box_rows x 64 columns.
cudaError_t map_2d(CUtensorMap* m, const void* p, int rows, int cols, int pitch, int box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(pitch) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
  return encode_bf16_map(m, p, 2, dims, strides, box);
}

// An MN-major operand: such a matrix in boxes of 64 rows (the sum's index) and 64 columns and, as far as
// whole blocks of 64 columns go (*solid columns), in boxes of `blocks` of them, block by block as the
// tensor core reads them: TMA takes about as long to start a box as to copy 4 KB. What follows the whole
// blocks is left to the first map, which has zeros past a row's end where the block map would read on.
// A row whose pitch has room for its last block may count it as whole: what it reads there ends in
// columns that are not stored.
cudaError_t map_mn(CUtensorMap* m, CUtensorMap* by_block, const void* p, int rows, int cols, int pitch, int blocks,
                   int* solid) {
  const int whole = pitch > cols ? (cols + 63) / 64 : cols / 64;
  *solid = 64 * whole;
  cudaError_t e = map_2d(m, p, rows, cols, pitch, 64);
  if (e != cudaSuccess || whole < blocks) {
    *solid = 0;
    return e;
  }
  const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(whole)};
  const uint64_t strides[2] = {static_cast<uint64_t>(pitch) * 2, 128};
  const uint32_t box[3] = {64, 64, static_cast<uint32_t>(blocks)};
  return encode_bf16_map(by_block, p, 3, dims, strides, box);
}

// How a launch is dealt out. The unit of cost is a 64-deep slice of a full tile (512 cycles, 0.27 us).
constexpr int kWorkers = 76;       // pairs of a GB300's 152 SMs
constexpr size_t kSlotBytes = static_cast<size_t>(kPairRows) * kAccCols * 4;
constexpr double kUnit = 6.0;      // slices that a tile costs beside its own: the ends of its pipeline
constexpr double kSumLaunch = 10;  // slices of the second launch of a cut plan
struct Plan {
  int width, tiles_m, tiles_n, tiles, direct, span, padded, slots;
  double cost;
};
// Tiles of `width` output columns (`full` at most). A slice of a narrow tile saves little: it still loads
// the 256 rows of A and goes round the ring. Measured against a full tile's: 0.84 at 80 of 128 columns,
// 0.90 at 112 of 128, 0.85 at 128 of 256 (1.05 at 192 and 1.0 at 64 of 256, where the halves of B do not
// start at a block: those widths are not offered).
Plan plan_width(int rows, int cols, int products, int nk, int width, int full, bool may_cut) {
  const double share = 0.65 + 0.35 * width / full;
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
  // time, and they meet in L2. Every pair's part is written and read once, together about 9 KB in a ns.
  int span = std::max(4, ceil_div(static_cast<long>(left) * nk, kWorkers)), padded = nk;
  if (2 * left <= kWorkers) {
    span = std::max(4, ceil_div(nk, kWorkers / left));
    padded = ceil_div(nk, span) * span;
  }
  const int pairs = ceil_div(static_cast<long>(left) * padded, span);
  const double bytes = static_cast<double>(pairs + left) * kPairRows * width * 8;
  const double cost = static_cast<double>(p.tiles / kWorkers) * (nk * share + kUnit) + span * share + 2 * kUnit +
                      kSumLaunch + bytes / 9000.0 / 270.0;
  if (cost < p.cost) {  // then nk > span: a share spans two tiles at most
    p.direct = p.tiles - left;
    p.span = span;
    p.padded = padded;
    p.cost = cost;
    p.slots = 2 * pairs;
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
// The others: 256 columns, or 128 where that saves a round.
Plan plan_sum(int rows, int cols, int products, int nk) {
  const Plan wide = plan_width(rows, cols, products, nk, 256, 256, true);
  const Plan narrow = plan_width(rows, cols, products, nk, 128, 256, true);
  return narrow.cost < 0.97 * wide.cost ? narrow : wide;
}
Plan plan_dx(int M, int N, int K, int terms) { return plan_sum(M, K, 1, terms * ceil_div(N, kBK)); }
Plan plan_dw(int M, int N, int K, int products) { return plan_sum(N, K, products, ceil_div(M, kBK)); }

// A problem of rows x cols outputs; `turn`: the pair that its numbers begin with.
Problem deal(const Plan& p, int rows, int cols, int nk0, int terms, int turn) {
  Problem q{};
  q.rows = rows;
  q.cols = cols;
  q.tiles_m = p.tiles_m;
  q.tiles_n = p.tiles_n;
  q.tiles = p.tiles;
  q.width = p.width;
  q.nk0 = nk0;
  q.nk = nk0 * terms;
  q.direct = p.direct;
  q.span = p.span;
  q.padded = p.padded;
  q.turn = turn;
  return q;
}
Problem no_problem() {
  Problem q{};
  q.span = q.padded = q.width = 1;
  return q;
}
// Pairs that a problem's last round keeps busy.
int last_round(const Plan& p) {
  if (p.direct == p.tiles) return p.tiles % kWorkers;
  return ceil_div(static_cast<long>(p.tiles - p.direct) * p.padded, p.span) % kWorkers;
}

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
  const bool cut = a.p[0].direct < a.p[0].tiles || a.p[1].direct < a.p[1].tiles;
  const int most = cut || a.p[1].tiles > 0 ? a.workers : std::min(a.workers, a.p[0].tiles);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(pairs, most)));
  cfg.numAttrs = after ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, a, maps);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t sum_parts(const GemmArgs& a, cudaStream_t stream) {
  const int cut0 = a.p[0].tiles - a.p[0].direct, cut1 = a.p[1].tiles - a.p[1].direct;
  if (cut0 + cut1 == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cut0 + cut1, std::max(cut0 > 0 ? a.p[0].width : 0, cut1 > 0 ? a.p[1].width : 0) / 16, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, part_sum_kernel, a, cut0);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// For one or two d_t [M, N] with w_t [N, K] and x [M, K]: dx [M, K] = sum_t d_t w_t and
// dw_t [N, K] = d_t^T x, dx or all dw's null where not wanted. d_t's rows are `pitch` elements apart.
cudaError_t run_grads(const void* const* d, int pitch, const void* const* w, int terms, const void* x, void* dx, void* const* dw,
                      int M, int N, int K, float* partial, bool after, uint32_t* dev_status, cudaStream_t stream) {
  GemmArgs a{};
  Maps m{};
  cudaError_t e = cudaSuccess;
  a.p[0] = a.p[1] = no_problem();
  int turn = 0, slot0 = 0;
  if (dx != nullptr) {
    const Plan plan = plan_dx(M, N, K, terms);
    Problem& p = a.p[0] = deal(plan, M, K, ceil_div(N, kBK), terms, 0);
    turn = last_round(plan);
    slot0 = plan.slots;
    p.out[0] = static_cast<__nv_bfloat16*>(dx);
    e = map_2d(&m.out[0][0], dx, M, K, K, 32);
    for (int t = 0; t < terms && e == cudaSuccess; ++t) {
      e = map_2d(&m.a[0][t], d[t], M, N, pitch, 128);
      if (e == cudaSuccess)
        e = map_mn(&m.b[0][t], &m.b_blocks[0][t], w[t], N, K, K, p.width / 128, &p.solid_b);
    }
  }
  if (dw[0] != nullptr && e == cudaSuccess) {
    Problem& p = a.p[1] = deal(plan_dw(M, N, K, terms), N, K, ceil_div(M, kBK), 1, turn);
    p.slot0 = slot0;
    e = map_mn(&m.b[1][0], &m.b_blocks[1][0], x, M, K, K, p.width / 128, &p.solid_b);
    for (int t = 0; t < terms && e == cudaSuccess; ++t) {
      p.out[t] = static_cast<__nv_bfloat16*>(dw[t]);
      e = map_mn(&m.a[1][t], &m.a_blocks[t], d[t], M, N, pitch, 2, &p.solid_a);
      if (e == cudaSuccess) e = map_2d(&m.out[1][t], dw[t], N, K, K, 32);
    }
  }
  if (e != cudaSuccess) return e;
  a.workers = kWorkers;
  a.partial = partial;
  a.dev_status = dev_status;
  e = launch<Use::Grads>(a, m, after, stream);
  return e != cudaSuccess ? e : sum_parts(a, stream);
}

// Outputs of `pitch` elements a row.
template <Use USE>
cudaError_t run_glu(const GluArgs& g, const void* dh, void* out0, void* out1, int pitch, cudaStream_t stream) {
  GemmArgs a{};
  a.p[0] = deal(plan_glu(g.M, g.F, g.K), g.M, g.F, ceil_div(g.K, kBK), 1, 0);
  a.p[1] = no_problem();
  a.workers = kWorkers;
  a.dh = static_cast<const __nv_bfloat16*>(dh);
  a.p[0].out[0] = static_cast<__nv_bfloat16*>(out0);
  a.p[0].out[1] = static_cast<__nv_bfloat16*>(out1);
  a.p[0].pitch = pitch;
  a.act = g.act;
  a.dev_status = g.dev_status;
  const int width = a.p[0].width;
  Maps m{};
  cudaError_t e = map_2d(&m.a[0][0], g.x, g.M, g.K, g.K, 128);
  if (e == cudaSuccess) e = map_2d(&m.b[0][0], g.w_gate, g.F, g.K, g.K, width);
  if (e == cudaSuccess) e = map_2d(&m.b[0][1], g.w_up, g.F, g.K, g.K, width);
  if (e == cudaSuccess && width == 128) {  // narrower tiles are stored by the threads
    e = map_2d(&m.out[0][0], out0, g.M, g.F, pitch, 32);
    if (e == cudaSuccess && USE == Use::GluGrad) e = map_2d(&m.out[0][1], out1, g.M, g.F, pitch, 32);
    if (e == cudaSuccess && USE == Use::GluGrad) e = map_2d(&m.dh, dh, g.M, g.F, g.F, 32);
  }
  return e != cudaSuccess ? e : launch<USE>(a, m, false, stream);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t grads_bytes(int M, int N, int K, int terms, bool dx, bool dw) {
  return static_cast<size_t>((dx ? plan_dx(M, N, K, terms).slots : 0) + (dw ? plan_dw(M, N, K, terms).slots : 0)) *
         kSlotBytes;
}

}  // namespace

cudaError_t launch_glu_fwd(const GluArgs& g, void* h, cudaStream_t stream) {
  if (g.M <= kGluDecodeRows) return launch_glu_decode(g, h, stream);
  return run_glu<Use::Glu>(g, nullptr, h, nullptr, g.F, stream);
}

// dg and du lie in rows of whole 64-column blocks: every box of them is aligned, and one brings two blocks.
int grad_pitch(int F) { return (F + 63) / 64 * 64; }
size_t glu_bwd_ws_bytes(int M, int F, int K, bool dx, bool dw) {
  return 2 * up256(static_cast<size_t>(M) * grad_pitch(F) * 2) + grads_bytes(M, F, K, 2, dx, dw);
}

cudaError_t launch_glu_bwd(const GluArgs& g, const void* dh, void* dx, void* dw_gate, void* dw_up, void* ws,
                           cudaStream_t stream) {
  const int pitch = grad_pitch(g.F);
  const size_t act = up256(static_cast<size_t>(g.M) * pitch * 2);
  void* dg = ws;
  void* du = static_cast<uint8_t*>(ws) + act;
  float* partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * act);
  const cudaError_t e = run_glu<Use::GluGrad>(g, dh, dg, du, pitch, stream);
  if (e != cudaSuccess) return e;
  const void* d[2] = {dg, du};
  const void* w[2] = {g.w_gate, g.w_up};
  void* dw[2] = {dw_gate, dw_up};
  return run_grads(d, pitch, w, 2, g.x, dx, dw, g.M, g.F, g.K, partial, true, g.dev_status, stream);
}

size_t linear_bwd_ws_bytes(int M, int N, int K, bool dx, bool dw) { return grads_bytes(M, N, K, 1, dx, dw); }

cudaError_t launch_linear_bwd(const void* dy, const void* x, const void* w, void* dx, void* dw, int M, int N, int K,
                              void* ws, uint32_t* dev_status, cudaStream_t stream) {
  return run_grads(&dy, N, &w, 1, x, dx, &dw, M, N, K, static_cast<float*>(ws), false, dev_status, stream);
}

}  // namespace rapt
