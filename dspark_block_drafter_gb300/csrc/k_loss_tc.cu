// The training loss of a bf16 head: its three products on the 5th-generation tensor cores.
//
//   logits  z[i][j]  = X[i] . [lm_head[j] | markov_w2[:, j]] + bias[j]      K = columns of X
//   dX      dx[i][c] = sum_j q[i][j] [lm_head | markov_w2^T][j][c]          K = head rows
//   dW      [d_lm_head | d_markov_w2^T][j][c] = scale sum_i q[i][j] X[i][c] K = rows
//
// i: compact rows, j: compact head rows, c: columns of X.  One kernel form does all three:
// a 128 (or, for a CTA pair, 256) x 256 tile of the result accumulates in TMEM over K-blocks
// of 64.  Every operand comes by TMA straight from the array it lies in, 64 elements of its
// contiguous index wide: a swizzled K-major tile when that index is K, a row of 64 x 64
// MN-major tiles when it is not, and the matrix descriptors say which.
// So no operand is ever transposed in memory, and the Markov term is nothing but some more
// K-blocks (logits) or columns (gradients), read from markov_w1's gathered rows and from
// markov_w2 as they are.
//
// Persistent and warp-specialised, one CTA per SM: warp 8 issues the TMA copies, one thread
// of warp 9 the MMAs; warps 0-3 take the first 128 columns of a finished accumulator, warps
// 4-7 the others (there are two accumulators, so that this overlaps the next products).
// Warp 10 writes the zeros of gradients that no product reaches (rows of masked tokens, of
// tokens that precede no slot): the logits and dX leave most of the memory bandwidth unused.
// (1.3 GB of them in the 448 x 2816 x 262144 head with 32768 rows in use: logits 90 -> 174 us,
// dX 70 -> 152 us, against 235 us by themselves.  dW, which writes, took twice as long.)
//
// The tensor core cuts each partial sum of an accumulator toward zero, so a long sum drifts:
// over K = 4352 the losses were off by 5e-6 of their size.  The logits' accumulator is
// therefore read every few K-blocks and the parts are added in fp32 registers (which hold the
// tile's 128 columns of a row until it is complete).  Pairs read it every 12 K-blocks (losses
// off by 5e-7, the logits of 4096 rows 6% slower than in one sum; every 8: 2e-7, 11%), single
// CTAs, which wait for memory anyway, every 4.  The gradients are rounded to bf16, and need such
// care only where a sum is long: each step of 16 loses near 1e-7 of a sum of terms of one sign
// (T = 2^20 rows: dW short by 0.6%; signs mixed, 0.1%).  dX adds to its partial result in memory
// every 1024 K-blocks, and dW sums more than 256 K-blocks in registers, in a kernel of its own
// (the registers cost the common case spills): a loss of 1e-4 in dW and 4e-4 in dX at most.
//
// 352 threads leave 168 registers each.  The logits' epilogue holds its 128 sums in them and spills a
// few others once a tile (single CTAs 60 words a thread, pairs 20; dX and dW in one launch 14, of more
// than 16384 rows 60): next to a tile's K loop, some thousand cycles, that does not show (without
// its 14 the joint launch takes the same 10.26 ms at 4096 rows).
//
// The logits are never stored.  Their epilogue has one row per thread: it takes the maximum
// and the sum of exponentials of each 128-column tile, the label's column aside, and, when
// gradients follow, stores how far each logit lies below its tile's maximum as a 16-bit
// fixed-point number (see loss.h), from which the gradient is made once the row's log-sum-exp
// is known.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "loss.h"
#include "ptx.cuh"

namespace dspark {

namespace {

constexpr int kTileM = 128, kTileN = 256, kBlockK = 64;
constexpr uint32_t kBox = 64 * 64 * 2;               // bytes of 64 rows of 64 elements
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 3);
constexpr uint32_t kRowBytes = 128;                  // dW: a row's part of a staged store
constexpr uint32_t kStaging = kEpiWarps * 32 * kRowBytes;
template <int CG>
constexpr int kSumBlocks = CG == 2 ? 12 : 4;         // K-blocks of one part of a logit's sum
constexpr int kDxBlocks = 1024;                      // K-blocks of one part of a sum of dX,
constexpr int kDwBlocks = 256;                       // and of dW where T is above that
constexpr int kSmemMax = 227 * 1024;
constexpr int kBarBytes = 512;
constexpr long long kWaitBudget = 2000000000ll;      // ~1 s of SM clocks

// (kGrads: dX and dW in one launch, each pair its units of the first, then of the second)
enum : int { kLogits = 0, kDx = 1, kDw = 2, kGrads = 3 };
// what the logits' epilogue makes: the statistics, the stored distances from the tile's
// maximum, or (with the log-sum-exp known) the gradient of the logits
enum : int { kWantStats = 1, kWantGap = 2, kWantGrad = 4 };

// The operands as a product reads them: A, B, and the Markov part's B of the logits or dX; A
// and B of dW.  K-major ones in one box a K-block, MN-major ones in one box of several
// 64-column chunks (or, where rows are not whole chunks, in one box for each chunk).
struct Maps {
  CUtensorMap a, b, b2, wa, wb;
};

// 256-column tiles of X's two parts that a gradient is computed for.
struct Columns {
  int head, markov;
  __host__ __device__ int all() const { return head + markov; }
};

struct TcArgs {
  LossPlan p;
  int v0, v1;          // compact head rows of this piece
  int want;            // kWant...
  int first;           // dX: the first piece (later ones add)
  Columns dx, dw;
  int chunked;         // dX: lm_head rows are whole 64-column chunks
  int zero0, zero1;    // the share of the plan's zeros this launch writes, in 1/64
};

constexpr int kZeroShare = 34;    // of the zeros the logits write, in 1/64; dX the others
constexpr int kRowGroup = 24;     // M tiles whose rows of X are kept in L2 together

// One unit of work: a tile of the result and a range of K-blocks.
struct Unit {
  int m, c0;           // first row (of M) and column (of N) of the tile
  int wide;            // its columns are 256, not 128
  bool markov, dw;
  int kb0, kb1;
  int split;
};

// The units of one CTA (or pair), in order.
template <int MODE, int CG>
struct Sequence {
  static constexpr int kRows = kTileM * CG;
  int me, ctas;                 // this CTA (pair) among all
  int mt, vt, nkb, tkb;         // row tiles, head-row tiles, K-blocks of head rows, of rows
  int splits, n_dx, n_dw;       // units of dX, dW
  int mine_dx, common, spare;   // kGrads: see below
  int Hp, Kx, units;
  Columns cx, cw;

  __device__ __forceinline__ Sequence(const TcArgs& g, int n_tok, int n_voc, int splits_, int me_,
                                      int ctas_)
      : me(me_), ctas(ctas_), splits(splits_), Hp(g.p.Hp), Kx(g.p.Kx), cx(g.dx), cw(g.dw) {
    const int cols = max(0, min(g.v1, n_voc) - g.v0);
    mt = (n_tok + kRows - 1) / kRows;
    vt = (cols + (MODE == kLogits ? kTileN : kRows) - 1) / (MODE == kLogits ? kTileN : kRows);
    nkb = (cols + kBlockK - 1) / kBlockK;
    tkb = loss_low(g.p, n_tok) && n_tok > 0 ? 2 * kLossLow / kBlockK
                                            : (n_tok + kBlockK - 1) / kBlockK;
    n_dx = mt * cx.all() * splits;
    n_dw = vt * cw.all();
    units = MODE == kLogits ? mt * vt : MODE == kDx ? n_dx : n_dw;
    if (MODE != kGrads) return;
    // dX first, in turn; `more` CTAs have one unit of it more than the others.  Then dW: the
    // first `common` rounds go to everyone, and the rest to those with fewer units of dX, so
    // that all end together.  Costs in 1/16 K-blocks: 12 blocks for a partial result of dX; a
    // tile of dW takes 11 at least (measured from 1 to 12 K-blocks: 6 to 13).
    const int more = n_dx % ctas;
    mine_dx = n_dx / ctas + (me < more ? 1 : 0);
    spare = ctas - more;
    common = (n_dw + ctas - 1) / ctas;
    if (more > 0) {
      // (in integers, so that every warp and CTA finds the same)
      const long long cost_x = 16ll * nkb / splits + 192, cost_w = max(16 * tkb + 32, 176);
      const long long each = (n_dx * cost_x + n_dw * cost_w) / ctas;
      const long long left = each - (n_dx / ctas + 1) * cost_x;
      // the rounds that fit before the average end, or one more: whichever ends first
      const int c = (int)min((long long)common, max(0ll, left / cost_w));
      auto end_of = [&](int rounds) {
        const long long rest = max(0ll, (long long)n_dw - (long long)rounds * ctas);
        return max(cost_x + rounds * cost_w, (rounds + (rest + spare - 1) / spare) * cost_w);
      };
      common = min(common, end_of(c) <= end_of(c + 1) ? c : c + 1);
    }
  }

  __device__ __forceinline__ Unit dx(int u) const {
    // splits of K in order, so that the CTAs at work share their operands' K range in L2
    Unit t;
    const int nt = cx.all();
    t.dw = false;
    t.split = u / (mt * nt);
    const int in = u % (mt * nt);
    t.m = in / nt * kRows;
    columns(t, cx, in % nt);
    t.kb0 = (int)((long long)nkb * t.split / splits);
    t.kb1 = (int)((long long)nkb * (t.split + 1) / splits);
    return t;
  }
  __device__ __forceinline__ Unit dw(int u) const {
    Unit t;
    const int nt = cw.all();
    t.dw = true;
    t.split = 0;
    t.m = u / nt * kRows;
    columns(t, cw, u % nt);
    t.kb0 = 0;
    t.kb1 = tkb;
    return t;
  }
  // N tile n: the head's columns, then the Markov part's; the last tile of a part may be narrow
  __device__ __forceinline__ void columns(Unit& t, const Columns& c, int n) const {
    t.markov = n >= c.head;
    t.c0 = t.markov ? Hp + (n - c.head) * kTileN : n * kTileN;
    t.wide = (t.markov ? Kx : Hp) - t.c0 > kTileN / 2;
  }
  __device__ __forceinline__ Unit logits(int u) const {
    // head-row tiles in order, all M tiles of a group for each: the head streams once for
    // every group
    Unit t;
    const int grp = u / (kRowGroup * vt), in = u - grp * kRowGroup * vt;
    const int rows = min(kRowGroup, mt - grp * kRowGroup);
    t.m = (grp * kRowGroup + in % rows) * kRows;
    t.c0 = in / rows * kTileN;
    t.wide = 1;
    t.markov = t.dw = false;
    t.kb0 = 0;
    t.kb1 = Kx / kBlockK;
    t.split = 0;
    return t;
  }

  // this CTA's i-th unit; false past the last
  __device__ __forceinline__ bool get(int i, Unit& t) const {
    if (MODE == kGrads) {
      if (i < mine_dx) {
        t = dx(me + i * ctas);
        return true;
      }
      const int j = i - mine_dx;
      int u = me + j * ctas;
      if (j >= common) {
        if (me < ctas - spare) return false;
        u = common * ctas + (j - common) * spare + me - (ctas - spare);
      }
      if (u >= n_dw) return false;
      t = dw(u);
      return true;
    }
    const int u = me + i * ctas;
    if (u >= units) return false;
    t = MODE == kLogits ? logits(u) : MODE == kDx ? dx(u) : dw(u);
    return true;
  }
};

template <int CG>
__device__ __forceinline__ void load_2d(uint8_t* dst, const CUtensorMap* m, uint64_t* bar,
                                        uint32_t bar_leader, int x, int y) {
  if (CG == 2)
    ptx::tma_load_2d_pair(dst, m, bar_leader, x, y);
  else
    ptx::tma_load_2d(dst, m, bar, x, y);
}
// columns [64 chunk, ...) of rows y ...
template <int CG>
__device__ __forceinline__ void load_chunks(uint8_t* dst, const CUtensorMap* m, uint64_t* bar,
                                            uint32_t bar_leader, int y, int chunk) {
  if (CG == 2)
    ptx::tma_load_3d_pair(dst, m, bar_leader, 0, y, chunk);
  else
    ptx::tma_load_3d(dst, m, bar, 0, y, chunk);
}

// This CTA's part of the zeros of a launch, by one warp.
template <int MODE>
__device__ __forceinline__ void write_zeros(const TcArgs& g, int lane) {
  const uint4 none = make_uint4(0, 0, 0, 0);
  const int parts = (int)gridDim.x, part = (int)blockIdx.x;
  for (int z = 0; z < g.p.n_zero; ++z) {
    const LossZero& q = g.p.zero[z];
    // items: rows, or 16-byte vectors (and the odd bytes, all fewer than 16, at the end)
    const long long items = q.keep ? (long long)(q.bytes / q.row_bytes) : (long long)(q.bytes / 16);
    const int z0 = q.early ? (MODE == kLogits ? 0 : 64) : g.zero0;
    const int z1 = q.early ? 64 : g.zero1;
    const long long lo = items * z0 / 64, n = items * z1 / 64 - lo;
    const long long a = lo + n * part / parts, b = lo + n * (part + 1) / parts;
    if (q.keep) {
      const int per = q.row_bytes / 16;
      for (long long r0 = a; r0 < b; r0 += 32) {
        unsigned m = __ballot_sync(0xFFFFFFFFu, r0 + lane < b && q.keep[r0 + lane] < 0);
        while (m) {
          uint4* row = reinterpret_cast<uint4*>(q.p) + (r0 + __ffs(m) - 1) * per;
          m &= m - 1;
          for (int k = lane; k < per; k += 32) row[k] = none;
        }
      }
    } else {
      uint4* v = reinterpret_cast<uint4*>(q.p);
#pragma unroll 4
      for (long long k = a + lane; k < b; k += 32) v[k] = none;
      if (z0 < 64 && z1 == 64 && part == 0 && lane < (int)(q.bytes % 16)) q.p[items * 16 + lane] = 0;
    }
  }
}

// LONG: the rows may be more than kDwBlocks K-blocks (kDw, kGrads).
template <int MODE, int CG, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
loss_product(const __grid_constant__ Maps maps, const __grid_constant__ TcArgs g, int stages) {
  constexpr int kBoxB = kTileN / CG / 64;              // boxes of N this CTA stages
  constexpr uint32_t kStageA = 2 * kBox, kStageB = kBoxB * kBox;
  constexpr uint32_t kStage = kStageA + kStageB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(smem + (size_t)stages * kStage);
  uint64_t* empty = full + stages;
  uint64_t* acc_full = empty + stages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  uint8_t* staging = smem + (size_t)stages * kStage + kBarBytes;   // dW only

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const LossPlan& p = g.p;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&acc_full[a], 1);
      ptx::mbar_init(&acc_empty[a], kEpiWarps * CG);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 0) {
    if (CG == 2) {
      ptx::tmem_alloc_pair(tmem_slot, 512);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(tmem_slot, 512);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t full0 = CG == 2 ? ptx::mapa_shared(ptx::smem_u32(full), 0) : 0;
  const uint32_t acc_empty0 = CG == 2 ? ptx::mapa_shared(ptx::smem_u32(acc_empty), 0) : 0;
  pdl_wait();
  pdl_signal();
  const int n_tok = (int)p.ctrl[kLossTok], n_voc = (int)p.ctrl[kLossVoc];
  const int splits = MODE == kDx || MODE == kGrads ? (int)p.ctrl[kLossSplits] : 1;
  const Sequence<MODE, CG> seq(g, n_tok, n_voc, splits, blockIdx.x / CG, gridDim.x / CG);
  // where the part of a unit's sum that starts at K-block kb ends
  auto part_end = [&](const Unit& t, int kb) {
    if (MODE == kLogits) return min(t.kb1, kb + kSumBlocks<CG>);
    if (MODE == kDx || (MODE == kGrads && !t.dw)) return min(t.kb1, kb + kDxBlocks);
    return LONG ? min(t.kb1, kb + kDwBlocks) : t.kb1;
  };

  auto give_up = [&]() {
    *abort_flag = 1;
    flag_error(p.ctrl, kErrTimeout);
  };

  if (warp == kEpiWarps) {
    // ---------------------------------------------------------------- producer
    // One thread issues every copy: what it does for a K-block has to take less time than
    // the block's MMAs (about 600 clocks).  With four 8 KB copies a block and the choice of
    // operands inside the loop, it bounded the logits and dX at 60% of the tensor pipe.
    if (lane == 0) {
      uint32_t it = 0, s = 0, ph = 0;
      bool ok = true;
      auto run = [&](int kb0, int kb1, auto fill) {
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          if (!ptx::mbar_wait(&empty[s], ph ^ 1, kWaitBudget, abort_flag)) {
            ok = false;
            return;
          }
          if (leader) ptx::mbar_arrive_expect_tx(&full[s], CG * kStage);
          uint8_t* a = smem + (size_t)s * kStage;
          fill(kb * kBlockK, a, a + kStageA, &full[s], full0 + s * 8);
          if (++s == (uint32_t)stages) {
            s = 0;
            ph ^= 1;
          }
        }
      };
      Unit t;
      for (int i = 0; ok && seq.get(i, t); ++i) {
        const int ma = t.m + (int)rank * kTileM;             // this CTA's rows of M
        const int half = (int)rank * (kTileN / CG) >> (t.wide ? 0 : 1);   // and its share of N
        if (MODE == kLogits) {
          const int v = g.v0 + t.c0 + half, hb = p.Hp / kBlockK;
          run(t.kb0, hb, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
            load_2d<CG>(a, &maps.a, bar, lead, k, ma);
            load_2d<CG>(b, &maps.b, bar, lead, k, v);
          });
          run(hb, t.kb1, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
            load_2d<CG>(a, &maps.a, bar, lead, k, ma);
#pragma unroll
            for (int j = 0; j < kBoxB; ++j)
              load_2d<CG>(b + j * kBox, &maps.b2, bar, lead, v + 64 * j, k - p.Hp);
          });
        } else if (MODE == kDw || (MODE == kGrads && t.dw)) {
          const int ca = ma / 64, cb = (t.c0 + half) / 64;
          run(t.kb0, t.kb1, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
            load_chunks<CG>(a, &maps.wa, bar, lead, k, ca);
            load_chunks<CG>(b, &maps.wb, bar, lead, k, cb);
          });
        } else {
          const int v0 = g.v0;
          if (t.markov) {
            const int c = t.c0 - p.Hp + half;
            run(t.kb0, t.kb1, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
              load_2d<CG>(a, &maps.a, bar, lead, k, ma);
              load_2d<CG>(b, &maps.b2, bar, lead, v0 + k, c);
            });
          } else if (g.chunked) {
            const int c = (t.c0 + half) / 64;
            run(t.kb0, t.kb1, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
              load_2d<CG>(a, &maps.a, bar, lead, k, ma);
              load_chunks<CG>(b, &maps.b, bar, lead, v0 + k, c);
            });
          } else {
            const int c = t.c0 + half;
            run(t.kb0, t.kb1, [&](int k, uint8_t* a, uint8_t* b, uint64_t* bar, uint32_t lead) {
              load_2d<CG>(a, &maps.a, bar, lead, k, ma);
#pragma unroll
              for (int j = 0; j < kBoxB; ++j)
                load_2d<CG>(b + j * kBox, &maps.b, bar, lead, c + 64 * j, v0 + k);
            });
          }
        }
      }
      if (!ok) {
        give_up();
        // let the copies already issued land before the CTA can exit
        if (CG == 1) {
          const uint32_t from = it > (uint32_t)stages ? it - stages : 0;
          for (uint32_t j = from; j < it; ++j)
            ptx::mbar_wait(&full[j % stages], (j / stages) & 1, kWaitBudget, nullptr);
        } else {
          const long long t0 = clock64();
          while (clock64() - t0 < 1000000) {
          }
        }
      }
    }
  } else if (warp == kEpiWarps + 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && leader) {
      uint32_t s = 0, ph = 0, local = 0;
      bool ok = true;
      const uint32_t base = ptx::smem_u32(smem);
      uint32_t d = 0, accum = 0;
      Unit t;
      auto run = [&](auto a_mn_c, auto b_mn_c, int blocks) {
        constexpr bool a_mn = decltype(a_mn_c)::value, b_mn = decltype(b_mn_c)::value;
        constexpr uint32_t wide = ptx::idesc_bf16_f32(kTileM * CG, kTileN, a_mn, b_mn);
        constexpr uint32_t narrow = ptx::idesc_bf16_f32(kTileM * CG, kTileN / 2, a_mn, b_mn);
        const uint32_t idesc = MODE == kLogits || t.wide ? wide : narrow;
        const uint64_t da0 = a_mn ? ptx::desc_mnmajor_sw128(base, kBox, 1024)
                                  : ptx::desc_kmajor_sw128(base);
        const uint64_t db0 = b_mn ? ptx::desc_mnmajor_sw128(base + kStageA, kBox, 1024)
                                  : ptx::desc_kmajor_sw128(base + kStageA);
        // 16 deep: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major box
        constexpr uint32_t sa = a_mn ? 128 : 2, sb = b_mn ? 128 : 2;
        for (int q = 0; q < blocks; ++q) {
          if (!ptx::mbar_wait(&full[s], ph, kWaitBudget, abort_flag)) {
            ok = false;
            return;
          }
          ptx::tc_fence_after();
          const uint64_t da = da0 + s * (kStage / 16), db = db0 + s * (kStage / 16);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k) {
            if (CG == 2)
              ptx::mma_f16_pair(d, da + k * sa, db + k * sb, idesc, k == 0 ? accum : 1u);
            else
              ptx::mma_f16(d, da + k * sa, db + k * sb, idesc, k == 0 ? accum : 1u);
          }
          accum = 1u;
          if (CG == 2)
            ptx::mma_commit_pair_multicast(&empty[s], 0x3);
          else
            ptx::mma_commit(&empty[s]);
          if (++s == (uint32_t)stages) {
            s = 0;
            ph ^= 1;
          }
        }
      };
      using Mn = std::true_type;
      using K = std::false_type;
      for (int i = 0; seq.get(i, t); ++i) {
        for (int kb = t.kb0, part = 0; part == 0 || kb < t.kb1; ++part, ++local) {
          const int end = part_end(t, kb);
          const uint32_t acc = local & 1, aph = (local >> 1) & 1;
          if (!ptx::mbar_wait(&acc_empty[acc], aph ^ 1, kWaitBudget, abort_flag)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          d = tmem + acc * kTileN;
          accum = 0u;
          if (MODE == kLogits) {
            // lm_head, then markov_w2
            const int head = max(0, min(end, p.Hp / kBlockK) - kb);
            run(K{}, K{}, head);
            if (ok) run(K{}, Mn{}, end - kb - head);
          } else if (MODE == kDw || (MODE == kGrads && t.dw)) {
            run(Mn{}, Mn{}, end - kb);
          } else if (t.markov) {
            run(K{}, K{}, end - kb);
          } else {
            run(K{}, Mn{}, end - kb);
          }
          kb = end;
          if (!ok) break;
          if (CG == 2)
            ptx::mma_commit_pair_multicast(&acc_full[acc], 0x3);
          else
            ptx::mma_commit(&acc_full[acc]);
        }
        if (!ok) break;
      }
      if (!ok) give_up();
      if (CG == 2)
        ptx::mma_commit_pair_multicast(drain, 0x1);
      else
        ptx::mma_commit(drain);
      ptx::mbar_wait(drain, 0, kWaitBudget, nullptr);
    }
  } else if (warp == kEpiWarps + 2) {
    if (MODE != kDw && g.zero1 > g.zero0) write_zeros<MODE>(g, lane);
  } else {
    // ---------------------------------------------------------------- epilogue
    const int quad = warp % 4, half = warp / 4;       // lanes and columns of this warp
    const uint32_t at0 = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
    const float scale = __uint_as_float(p.ctrl[kLossScale]);
    uint32_t local = 0;
    bool ok = true;
    // the local-th accumulator is complete / has been read
    auto acc_wait = [&]() {
      ok = __all_sync(0xFFFFFFFFu, ptx::mbar_wait(&acc_full[local & 1], (local >> 1) & 1,
                                                  kWaitBudget, abort_flag));
      if (!ok) give_up();
      ptx::tc_fence_after();
      return ok;
    };
    auto acc_free = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2)
          // (not a cluster-wide release: that waits for the last tile's stores, and held the
          // next products up by half their time when K is short)
          ptx::mbar_arrive_cluster_tmem(acc_empty0 + (local & 1) * 8);
        else
          ptx::mbar_arrive(&acc_empty[local & 1]);
      }
      ++local;
    };
    Unit t;
    for (int i = 0; ok && seq.get(i, t); ++i) {
      const int m = t.m + (int)rank * kTileM + quad * 32 + lane;   // this thread's row of M
      if (MODE == kLogits) {
        const bool live = m < n_tok;
        // (the low rows of q: written with their rows' gradients, before that zeros)
        const bool low = (g.want & kWantGrad) && loss_low(p, n_tok);
        const bool mine = !low || live || (m < kLossLow || m >= kLossLow + n_tok);
        const int lab = live ? p.lab[m] : -1;
        const int v0 = g.v0 + t.c0 + half * 128;             // compact head row of column 0
        const int n_in = n_voc - v0;                          // columns that exist
        float z[128];
        for (int kb = t.kb0; kb < t.kb1; kb += kSumBlocks<CG>) {
          if (!acc_wait()) break;
          const uint32_t at = at0 + (local & 1) * kTileN;
          const bool first = kb == t.kb0;
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(at + c, r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              z[c + j] = first ? __uint_as_float(r[j]) : z[c + j] + __uint_as_float(r[j]);
          }
          acc_free();
        }
        if (!ok) break;
        if (p.vlist) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j < n_in) z[j] += __ldg(p.biasc + v0 + j);
        }
        if (n_in < 128) {
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (j >= n_in) z[j] = -INFINITY;
        }
        const bool here = lab >= v0 && lab < v0 + 128;
        if ((g.want & kWantStats) && __any_sync(0xFFFFFFFFu, here)) {
          float zl = 0.f;                         // the label's logit
#pragma unroll
          for (int j = 0; j < 128; ++j)
            if (lab == v0 + j) {                  // (kept out of the statistics)
              zl = z[j];
              z[j] = -INFINITY;
            }
          if (here) p.zlab[m] = zl;
        }
        float ref = 0.f, wt = 0.f;
        if (g.want & kWantStats) {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 128; ++j) mx[j % 4] = fmaxf(mx[j % 4], z[j]);
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          ref = top > -INFINITY ? top : 0.f;      // (a NaN passes the maximum, not the sum)
          float sum[4] = {};
#pragma unroll
          for (int j = 0; j < 128; ++j) sum[j % 4] += loss_exp(z[j] - ref);
          if (live && n_in > 0)
            p.stat[(size_t)m * p.n_stat + v0 / 128] =
                make_float2(top, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        } else if (live) {
          ref = p.lse[m];
          wt = p.wrow[m];
        }
        if (g.want & (kWantGap | kWantGrad)) {
          uint16_t* qrow = (uint16_t*)p.q + (size_t)m * p.ldq + (v0 - g.v0);
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[8], l[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float d0 = z[c + j] - ref, d1 = z[c + j + 1] - ref;
              if (g.want & kWantGrad) {
                const float e0 = wt * loss_exp(d0), e1 = wt * loss_exp(d1);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(e0, e1);
                o[j / 2] = *reinterpret_cast<const uint32_t*>(&b2);
                if (CG == 1) {
                  const __nv_bfloat162 l2 =
                      __floats2bfloat162_rn(e0 - __low2float(b2), e1 - __high2float(b2));
                  l[j / 2] = *reinterpret_cast<const uint32_t*>(&l2);
                }
              } else {
                o[j / 2] = __byte_perm(loss_gap(-d0), loss_gap(-d1), 0x5410);
              }
              if (!live) o[j / 2] = 0u;
            }
            if (CG == 2 || mine) ptx::st_global_v8(qrow + c, o);
            if (CG == 1 && low && live) ptx::st_global_v8(qrow + kLossLow * p.ldq + c, l);
          }
          if ((g.want & kWantGrad) && here)       // (after this thread's vector store)
            loss_put_label(p, m, CG == 1 && low, reinterpret_cast<__nv_bfloat16*>(qrow) + (lab - v0),
                           loss_label_entry(wt, p.loss[p.tok[m]]));
        }
      } else {
        const bool none = t.kb1 <= t.kb0;             // (nothing was accumulated)
        const bool markov = t.markov;
        const int c0 = t.c0 + half * 128;
        if (MODE == kDx || (MODE == kGrads && !t.dw)) {
          const int width = min(128, (markov ? p.Kx : p.Hp) - c0);
          float* dx = p.dxp + ((size_t)t.split * loss_split_rows(n_tok) + m) * p.Kx + c0;
          bool add = !g.first;
          for (int kb = t.kb0, end; ok; kb = end, add = true) {
            end = part_end(t, kb);
            if (!acc_wait()) break;
            const uint32_t at = at0 + (local & 1) * kTileN;
#pragma unroll 1
            for (int c = 0; c < width; c += 32) {
              uint32_t r[32];
              ptx::tmem_ld_32x32b_x32(at + c, r);
              ptx::tmem_ld_wait();
              if (m >= n_tok &&
                  !(CG == 1 && loss_low(p, n_tok) && m >= kLossLow && m < kLossLow + n_tok))
                continue;
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                float x[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) x[b] = none ? 0.f : __uint_as_float(r[j + b]);
                if (add) {
                  const float4 y0 = *reinterpret_cast<const float4*>(dx + c + j);
                  const float4 y1 = *reinterpret_cast<const float4*>(dx + c + j + 4);
                  x[0] += y0.x; x[1] += y0.y; x[2] += y0.z; x[3] += y0.w;
                  x[4] += y1.x; x[5] += y1.y; x[6] += y1.z; x[7] += y1.w;
                }
                ptx::st_global_v8(dx + c + j, x);
              }
            }
            acc_free();
            if (end >= t.kb1) break;
          }
          if (!ok) break;
        } else {
          const int j0 = g.v0 + m;                            // compact head row
          const bool live = j0 < min(g.v1, n_voc);
          const size_t row = live ? (size_t)loss_head_row(p, j0) : 0;
          const int width = min(128, markov ? p.r - (c0 - p.Hp) : p.H - c0);
          float z[LONG ? 128 : 1];                            // the parts before the last
          if (LONG) {
#pragma unroll
            for (int c = 0; c < 128; ++c) z[c] = 0.f;
            for (int kb = t.kb0, end = part_end(t, kb); end < t.kb1; kb = end, end = part_end(t, kb)) {
              if (!acc_wait()) break;
              const uint32_t at = at0 + (local & 1) * kTileN;
#pragma unroll
              for (int c = 0; c < 128; c += 32) {
                uint32_t r[32];
                ptx::tmem_ld_32x32b_x32(at + c, r);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) z[c + j] += __uint_as_float(r[j]);
              }
              acc_free();
            }
            if (!ok) break;
          }
          if (!acc_wait()) break;
          const uint32_t at = at0 + (local & 1) * kTileN;
          uint32_t o[64];                                     // 128 columns, in pairs
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(at + c, r);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float x0 = __uint_as_float(r[j]), x1 = __uint_as_float(r[j + 1]);
              if (LONG) {
                x0 += z[c + j];
                x1 += z[c + j + 1];
              }
              const __nv_bfloat162 b2 =
                  __floats2bfloat162_rn(none ? 0.f : x0 * scale, none ? 0.f : x1 * scale);
              o[(c + j) / 2] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
          acc_free();
          if (markov) {
            // column by column: a warp's rows are neighbours there
            uint16_t* d = (uint16_t*)p.d_w2 + (size_t)(c0 - p.Hp) * p.Vh + row;
            if (p.vlist) {
#pragma unroll
              for (int j = 0; j < 128; ++j)
                if (live && j < width)
                  d[(size_t)j * p.Vh] = (uint16_t)(j & 1 ? o[j / 2] >> 16 : o[j / 2] & 0xFFFFu);
            } else {
              // lanes in pairs: the even one stores both rows of the even column, the odd one
              // those of the odd column (V_head is a multiple of 8, so both rows exist)
              const int odd = lane & 1;
              d -= odd;
#pragma unroll
              for (int q = 0; q < 64; ++q) {
                const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, o[q], 1);
                const uint32_t both = odd ? __byte_perm(other, o[q], 0x7632)
                                          : __byte_perm(o[q], other, 0x5410);
                if (live && 2 * q + odd < width)
                  *reinterpret_cast<uint32_t*>(d + (size_t)(2 * q + odd) * p.Vh) = both;
              }
            }
          } else {
            // through shared memory, so that eight lanes store 128 bytes of one row (one
            // row a lane, 16 bytes at a time, reached a fifth of the write bandwidth)
            uint8_t* st = staging + warp * 32 * kRowBytes;
#pragma unroll
            for (int c = 0; c < 128; c += 64) {
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(st + lane * kRowBytes + ((q ^ (lane & 7)) << 4)) =
                    make_uint4(o[c / 2 + 4 * q], o[c / 2 + 4 * q + 1], o[c / 2 + 4 * q + 2],
                               o[c / 2 + 4 * q + 3]);
              __syncwarp();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const int rr = 4 * q + lane / 8, ch = lane & 7, col = c + 8 * ch;
                const uint4 v =
                    *reinterpret_cast<const uint4*>(st + rr * kRowBytes + ((ch ^ (rr & 7)) << 4));
                const int to = __shfl_sync(0xFFFFFFFFu, live ? (int)row : -1, rr);
                if (to >= 0 && col < width)                   // (H is a multiple of 8)
                  *reinterpret_cast<uint4*>((__nv_bfloat16*)p.d_lm_head + (size_t)to * p.H + c0 +
                                            col) = v;
              }
            }
          }
        }
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  if (warp == 0) {
    ptx::tc_fence_after();
    if (CG == 2)
      ptx::tmem_dealloc_pair(tmem, 512);
    else
      ptx::tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
  });
  return fn;
}

// A [rows][ld] bf16 array, `cols` of each row in use, read 64 columns x `high` rows at a time
// (zeros outside).
bool map_2d(CUtensorMap* m, const void* base, size_t cols, size_t rows, size_t ld, int high) {
  auto encode = encode_fn();
  if (!encode) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)high}, es[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)base, dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same as (64 columns, row, chunk of 64 columns), read 64 rows x `chunks` chunks at a
// time; rows are whole chunks.
bool map_chunks(CUtensorMap* m, const void* base, size_t cols, size_t rows, int chunks) {
  auto encode = encode_fn();
  if (!encode || cols % 64) return false;
  cuuint64_t dims[3] = {64, rows, cols / 64}, strides[2] = {cols * 2, 128};
  cuuint32_t box[3] = {64, 64, (cuuint32_t)chunks}, es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)base, dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int CG>
bool make_maps(const TcArgs& g, Maps* m) {
  const LossPlan& p = g.p;
  constexpr int share = kTileN / CG;                   // rows of N a CTA stages
  const void* w = p.wc ? p.wc : p.lm_head;
  const void* w2 = p.wc ? p.w2c : p.w2;
  bool ok = true;
  if (MODE == kLogits) {
    ok = map_2d(&m->a, p.x, p.Kx, p.Tp, p.Kx, kTileM) && map_2d(&m->b, w, p.H, p.Vh, p.H, share);
    m->b2 = m->b;
    if (p.r > 0) ok = ok && map_2d(&m->b2, w2, p.Vh, p.r, p.Vh, 64);
  }
  if (MODE == kDx || MODE == kGrads) {
    ok = map_2d(&m->a, p.q, p.ldq, p.Tp, p.ldq, kTileM) &&
         (g.chunked ? map_chunks(&m->b, w, p.H, p.Vh, share / 64)
                    : map_2d(&m->b, w, p.H, p.Vh, p.H, 64));
    m->b2 = m->b;
    if (p.r > 0) ok = ok && map_2d(&m->b2, w2, p.Vh, p.r, p.Vh, share);
  }
  if (MODE == kDw || MODE == kGrads)
    ok = ok && map_chunks(&m->wa, p.q, p.ldq, p.Tp, kTileM / 64) &&
         map_chunks(&m->wb, p.x, p.Kx, p.Tp, share / 64);
  return ok;
}

template <int MODE, int CG, bool LONG = false>
cudaError_t launch(const TcArgs& g, long long tiles) {
  if (tiles <= 0) return cudaSuccess;
  Maps maps = {};
  if (!make_maps<MODE, CG>(g, &maps)) return cudaErrorInvalidValue;
  constexpr uint32_t stage = 2 * kBox + kTileN / CG / 64 * kBox;
  constexpr uint32_t fixed = 1024 + kBarBytes + (MODE == kDw || MODE == kGrads ? kStaging : 0);
  constexpr int stages = (kSmemMax - fixed) / stage;
  constexpr size_t smem = fixed + (size_t)stages * stage;
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = raise_smem_limit((const void*)loss_product<MODE, CG, LONG>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(tiles, std::max(1, sms / CG)) * CG);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = g.p.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, loss_product<MODE, CG, LONG>, maps, g, stages);
}

// Single CTAs (128-row tiles) when the rows fit one tile, pairs (256) otherwise.
bool single(int T) { return T <= kTileM; }

int row_tiles(int T) { return (T + 255) / 256; }   // (one tile of either height up to 128)

}  // namespace

// The most splits of the vocabulary that loss_pick_splits may take: eight units for each CTA
// (or pair), at least 6.
int loss_tc_splits(int T, int Hp, int rp) {
  const int tiles = row_tiles(T) * ((Hp + kTileN - 1) / kTileN + (rp + kTileN - 1) / kTileN);
  const int units = single(T) ? 152 : 76;
  return std::max(6, std::min(64, (8 * units + tiles - 1) / std::max(1, tiles)));
}

cudaError_t launch_loss_logits_tc(const LossPlan& p, int v0, int v1, bool stats, bool store) {
  TcArgs g{};
  g.p = p;
  g.v0 = v0;
  g.v1 = v1;
  g.want = stats ? kWantStats | (store ? kWantGap : 0) : kWantGrad;
  if (stats && p.n_zero > 0) g.zero1 = p.d_hidden || p.d_w1 ? kZeroShare : 64;
  const long long tiles = (long long)row_tiles(p.T) * ((v1 - v0 + kTileN - 1) / kTileN);
  return single(p.T) ? launch<kLogits, 1>(g, tiles) : launch<kLogits, 2>(g, tiles);
}

// The two gradient products of columns [v0, v1), in one launch of pairs where both are asked
// for: alone, each leaves pairs without work at its end (four pieces of 1001 rows 493 -> 421 us for
// the whole call; the frozen head with 512 rows 1050 us, 4096 rows 9.8 ms, either way).
cudaError_t launch_loss_grads_tc(const LossPlan& p, int v0, int v1, bool first) {
  TcArgs g{};
  g.p = p;
  g.v0 = v0;
  g.v1 = v1;
  g.first = first;
  g.chunked = p.H % 64 == 0;
  const int head = (p.Hp + kTileN - 1) / kTileN, markov = (p.rp + kTileN - 1) / kTileN;
  g.dx = {p.d_hidden ? head : 0, p.d_w1 ? markov : 0};
  g.dw = {p.d_lm_head ? head : 0, p.d_w2 ? markov : 0};
  if (first && p.n_zero > 0 && g.dx.all() > 0) {
    g.zero0 = kZeroShare;
    g.zero1 = 64;
  }
  const long long n_dx = (long long)row_tiles(p.T) * g.dx.all() * p.splits;
  const long long n_dw = (long long)((v1 - v0 + 255) / 256) * g.dw.all();
  const bool lengthy = p.T > kDwBlocks * kBlockK;
  if (n_dx > 0 && n_dw > 0 && !single(p.T))
    return lengthy ? launch<kGrads, 2, true>(g, n_dx + n_dw) : launch<kGrads, 2>(g, n_dx + n_dw);
  cudaError_t e = single(p.T) ? launch<kDx, 1>(g, n_dx) : launch<kDx, 2>(g, n_dx);
  if (e == cudaSuccess) e = lengthy ? launch<kDw, 2, true>(g, n_dw) : launch<kDw, 2>(g, n_dw);
  return e;
}

}  // namespace dspark
