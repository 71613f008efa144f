// sq_grouped.cu -- 8-bit linears whose rows are grouped by expert, and the
// block-scaled E4M3 linear, on the 5th-generation tensor cores (sm_100a).
//
// Rows offsets[e] .. offsets[e+1] of Xq are multiplied by expert e's
// weights Wq[e] ([N][K]); the dense block-scaled linear is one group of all
// rows.  Three ways codes are scaled:
//   I8, E4M3   y_tn = ((float)sum_j xq wq * dx_t) * dw_en
//   Block      y_tn = sum_b (dx_tb dw_e,n/128,b) * sum_{j in b} xq wq
// For Block the tensor cores sum one block of 128 channels at a time into
// TMEM, and the epilogue warps add it, times its scale, into fp32 registers:
// a fused multiply-add per (row, column, block), each block's product summed
// in fp32 before it is scaled.
//
// The groups' sizes stay on the device: each CTA reads the offsets and forms
// the prefix sums of the groups' tile counts, and tiles are numbered over
// all groups.
//
// Times in this file's comments are per call in a captured graph that takes
// three sets of inputs in turn (weights of up to some 40 MB then come from L2),
// both sides of one change on one device.  Long runs of the large shapes are
// 10 to 15 % slower, under the power limit.
#include "sq_capacity.h"
#include "sq_common.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kBlk = 128;          // channels per scale block = K bytes per stage
// Warps 0 and 2 load Xq and Wq, warp 1 issues the MMAs, warp 3 works out the
// split tiles (idle with pairs), then eight epilogue warps.
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStageBytes = 4096;  // an epilogue warp's output staging: 32 rows x 128 bytes

// One 128-channel block's MMAs (four of K = 32), the commit on `done` (of both
// CTAs for a pair), and whether the barriers of the next step, `full` and
// `tempty`, have completed their phases: asked for before the MMAs are issued
// and looked at after the commit, behind the MMAs.  The whole warp runs this
// and an elected lane issues: descriptors are then warp-uniform values, which
// the MMAs take from uniform registers (one lane alone: about 290 cycles to
// issue a block, so 103).
struct Seen {
  uint32_t full, tempty;
};
#define SQ_MMA4(GROUP, KIND, COMMIT)                                                              \
  "{\n\t.reg .pred one, first, add, pf, pt;\n\t.reg .b64 a, b;\n\t"                               \
  "elect.sync _|one, 0xffffffff;\n\t"                                                            \
  "setp.ne.b32 first, %6, 0;\n\tsetp.eq.b32 add, 0, 0;\n\t"                                      \
  "mbarrier.test_wait.parity.shared::cta.b64 pf, [%8], %9;\n\t"                                  \
  "mbarrier.test_wait.parity.shared::cta.b64 pt, [%10], %11;\n\t"                                \
  "@one tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%2], %3, %4, %5, first;\n\t"            \
  "add.s64 a, %3, 2;\n\tadd.s64 b, %4, 2;\n\t"                                                  \
  "@one tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%2], a, b, %5, add;\n\t"                \
  "add.s64 a, %3, 4;\n\tadd.s64 b, %4, 4;\n\t"                                                  \
  "@one tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%2], a, b, %5, add;\n\t"                \
  "add.s64 a, %3, 6;\n\tadd.s64 b, %4, 6;\n\t"                                                  \
  "@one tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%2], a, b, %5, add;\n\t" COMMIT         \
  "selp.u32 %0, 1, 0, pf;\n\tselp.u32 %1, 1, 0, pt;\n\t}\n"
#define SQ_COMMIT1 "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t"
// one instruction for both CTAs
#define SQ_COMMIT2                                                                                     \
  ".reg .b16 both;\n\tmov.b16 both, 3;\n\t"                                                            \
  "@one tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], both;\n\t"
#define SQ_MMA4_ARGS                                                                                          \
  : "=r"(seen.full), "=r"(seen.tempty)                                                                        \
  : "r"(d), "l"(a0), "l"(b0), "r"(idesc), "r"(add), "r"(smem_u32(done)), "r"(smem_u32(full)), "r"(full_parity), \
    "r"(smem_u32(tempty)), "r"(tempty_parity)                                                                 \
  : "memory"
template <int CG, bool F8>
__device__ __forceinline__ Seen mma_block(uint32_t d, uint64_t a0, uint64_t b0, uint32_t idesc, uint32_t add,
                                          uint64_t *done, uint64_t *full, uint32_t full_parity, uint64_t *tempty,
                                          uint32_t tempty_parity) {
  Seen seen;
  if constexpr (CG == 1 && F8) {
    asm volatile(SQ_MMA4("1", "f8f6f4", SQ_COMMIT1) SQ_MMA4_ARGS);
  } else if constexpr (CG == 1) {
    asm volatile(SQ_MMA4("1", "i8", SQ_COMMIT1) SQ_MMA4_ARGS);
  } else if constexpr (F8) {
    asm volatile(SQ_MMA4("2", "f8f6f4", SQ_COMMIT2) SQ_MMA4_ARGS);
  } else {
    asm volatile(SQ_MMA4("2", "i8", SQ_COMMIT2) SQ_MMA4_ARGS);
  }
  return seen;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Arrive on an mbarrier of another CTA of the cluster (shared::cluster
// address).  Without .release.cluster, which waits for the thread's earlier
// global stores: the TMEM reads that it publishes are ordered by
// tcgen05.wait::ld and the tcgen05 fences (per-block releases of the pair
// kernel, 4096 x 11008 x 4096: 365 -> 223 us).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Arrive once on the mbarrier at this address in both CTAs of the pair when
// the MMAs issued so far have completed.
__device__ __forceinline__ void umma_commit_both(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// The MMA warp's loop, for both kernels: n blocks of 128 channels, `left` of
// them to the end of the first tile and nk in every later one.  One warp's
// waits, issues and commits bound it, so the ring's stages are unrolled and a
// block whose operands are there costs one vote besides its MMAs (with the
// elected issue, 4096 x 11008 x 4096: INT8 128 -> 115 us, E4M3 144 -> 128,
// block scales 195 -> 176).  kBlock: every block has an accumulator of its
// own; otherwise a tile has one, handed over on tfull (with block scales on
// the stage's own barrier).  Ends early when a wait runs out.
template <int CG, bool F8, bool kBlock, int kStages, int kBufs, uint32_t kA, uint32_t kB, int kCols>
__device__ __forceinline__ void mma_loop(uint32_t sA, uint32_t sB, uint64_t *full, uint64_t *empty, uint64_t *tfull,
                                         uint64_t *tempty, uint32_t tmem, uint32_t idesc, int64_t n, int nk, int left,
                                         volatile int *abort, unsigned *err) {
  const uint64_t a0 = desc_sw128_kmajor(sA), b0 = desc_sw128_kmajor(sB);
  uint32_t phase = 0, buf = 0, bphase = 1;
  bool first = true;
  Seen seen = {0u, 0u};
#pragma unroll 1
  for (;; phase ^= 1) {
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
      if (n == 0) return;
      --n;
      const bool last = kBlock || left == 1 || n == 0;
      if (!__all_sync(0xffffffffu, seen.full && (!first || seen.tempty))) {
        if (!__all_sync(0xffffffffu, (!first || mbar_wait(&tempty[buf], bphase, abort, err)) &&
                                         mbar_wait(&full[st], phase, abort, err)))
          return;
      }
      tc_fence_after();
      const uint32_t d = tmem + buf * kCols, add = kBlock || first ? 0u : 1u;
      uint64_t *const done = tfull + buf;
      if (last && ++buf == kBufs) {
        buf = 0;
        bphase ^= 1;
      }
      const int next = (st + 1) % kStages;
      seen = mma_block<CG, F8>(d, a0 + st * (kA >> 4), b0 + st * (kB >> 4), idesc, add, &empty[st], &full[next],
                               phase ^ (next == 0 ? 1u : 0u), &tempty[buf], bphase);
      if (!kBlock && last && elect_one()) {
        if constexpr (CG == 2) {
          umma_commit_both(done);
        } else {
          umma_commit(done);
        }
      }
      first = last;
      if (!kBlock && --left == 0) left = nk;
    }
  }
}

// ---------------------------------------------------------------------------
// The groups' table in shared memory: row[e] = first row of group e (row[E]
// the end of the last), tile[e] = tiles of the groups before e.  Offsets are
// clamped to [0, T] and made non-decreasing by a running maximum, so no
// input leads to a row outside [0, T).  Ends with a block barrier.
// ---------------------------------------------------------------------------
struct Groups {
  int *row, *tile;
};

__device__ __forceinline__ int ceil_div_dev(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ void build_groups(const Groups &g, const int32_t *__restrict__ offsets, int E, int T,
                                             int tile_rows, int ntn) {
  if (offsets == nullptr) {
    if (threadIdx.x == 0) {
      g.row[0] = 0;
      g.row[1] = T;
      g.tile[0] = 0;
      g.tile[1] = ceil_div_dev(T, tile_rows) * ntn;
    }
  } else {
    for (int i = threadIdx.x; i <= E; i += blockDim.x) g.row[i] = min(max(__ldg(offsets + i), 0), T);
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int top = 0, sum = 0;
      for (int base = 0; base <= E; base += 32) {
        const int i = base + lane;
        int v = i <= E ? g.row[i] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v = max(v, u);
        }
        v = max(v, top);
        int prev = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) prev = i == 0 ? v : top;
        int t = ceil_div_dev(v - prev, tile_rows) * ntn;  // tiles of group i - 1
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, t, o);
          if (lane >= o) t += u;
        }
        t += sum;
        if (i <= E) {
          g.row[i] = v;
          g.tile[i] = t;
        }
        top = __shfl_sync(0xffffffffu, v, 31);
        sum = __shfl_sync(0xffffffffu, t, 31);
      }
    }
  }
  __syncthreads();
}

// Division by d, for dividends below 2^31: with 2^(l-1) < d <= 2^l and
// m = floor(2^(31+l) / d) + 1, m d exceeds 2^(31+l) by at most d <= 2^l, so
// w m / 2^(31+l) exceeds w / d by less than 1 / d and has the same floor.
// (An integer division is some 100 cycles, and several in a row held back a
// CTA's first load.)
struct FastDiv {
  uint32_t d, m, shift;
  explicit FastDiv(uint32_t div) : d(div), shift(31) {
    while ((1u << (shift - 31)) < d) ++shift;
    m = (uint32_t)((1ull << shift) / d + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t w) const { return (uint32_t)((uint64_t)w * m >> shift); }
};

// Where a tile lies; find() starts from the group of the tile before.
struct Place {
  int e = 0, row0 = 0, rows = 0, mb = 0, nb = 0;
  __device__ __forceinline__ void find(const Groups &g, int E, int tile, int tile_rows) {
    if (tile < g.tile[e]) e = 0;
    if (tile >= g.tile[e + 1]) {  // the first group that ends beyond the tile
      int lo = e + 1, hi = E - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tile < g.tile[mid + 1]) {
          hi = mid;
        } else {
          lo = mid + 1;
        }
      }
      e = lo;
    }
    row0 = g.row[e];
    rows = g.row[e + 1] - row0;
    const int nm = ceil_div_dev(rows, tile_rows), local = tile - g.tile[e];
    nb = nm == 1 ? local : local / nm;
    mb = local - nb * nm;
  }
};

// ---------------------------------------------------------------------------
// Output: a warp holds 32 rows, one per lane, and hands over their columns
// in order, 32 at a time.  They pass through 32 x 128 bytes of its own shared
// memory (16-byte chunks swizzled by row: conflict-free both ways) so that
// global stores write whole 128-byte rows.
// ---------------------------------------------------------------------------
template <OutKind KIND>
struct RowStore {
  static constexpr int kEsz = KIND == OutKind::F32 ? 4 : 2;
  uint8_t *stage;
  uint8_t *y;
  int64_t ldy;
  int row0, row_end, N, lane;

  // v: columns n0 .. n0 + 31 of this lane's row; n0 % 32 == 0
  __device__ __forceinline__ void put(const float (&v)[32], int n0) {
    if constexpr (KIND == OutKind::F32) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        chunk(c) = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                              __float_as_uint(v[4 * c + 3]));
      flush(n0);
    } else {
      const int half = (n0 / 32) & 1;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (KIND == OutKind::BF16) {
            __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
            p[i] = *reinterpret_cast<uint32_t *>(&h);
          } else {
            __half2 h = __floats2half2_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
            p[i] = *reinterpret_cast<uint32_t *>(&h);
          }
        }
        chunk(half * 4 + c) = make_uint4(p[0], p[1], p[2], p[3]);
      }
      if (half == 1) flush(n0 - 32);
    }
  }

 private:
  __device__ __forceinline__ uint4 &chunk(int c) {
    return *reinterpret_cast<uint4 *>(stage + lane * 128 + ((c ^ (lane & 7)) << 4));
  }
  __device__ __forceinline__ void flush(int n0) {
    __syncwarp();
    const int c = lane & 7, n = n0 + c * (16 / kEsz);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (row0 + r < row_end && n < N)
        *reinterpret_cast<uint4 *>(y + ((int64_t)(row0 + r) * ldy + n) * kEsz) =
            *reinterpret_cast<const uint4 *>(stage + r * 128 + ((c ^ (r & 7)) << 4));
    }
    __syncwarp();
  }
};

constexpr int kPairRows = 256, kPairCols = 256;
struct PairTileSmem {
  static constexpr int kStages = 5;
  static constexpr uint32_t kA = 128 * kBlk;        // this CTA's rows of Xq
  static constexpr uint32_t kB = (kPairCols / 2) * kBlk;  // this CTA's half of the tile's rows of Wq
  static constexpr uint32_t kRing = kStages * (kA + kB);
  static constexpr uint32_t kStaging = kEpiWarps * kStageBytes;
  static constexpr uint32_t kTable = 2 * (kMaxExperts + 1) * 4 + 8;
  static constexpr uint32_t kBars = (2 * kStages + 5) * 8 + 16;
  static constexpr uint32_t kTotal = kRing + kStaging + kTable + kBars + 1024;
};

// Registers are handed from the first warpgroup to the two epilogue ones,
// which hold a 128-column row of fp32 sums per thread: 384 threads launch with
// 168 each, and 104 + 2 * 200 = 3 * 168.
__device__ __forceinline__ void regs_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }
__device__ __forceinline__ void regs_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 200;"); }

// Persistent over 256 x 256 tiles of Y: a pair of CTAs works on one tile
// (tcgen05 cta_group::2), each with 128 rows of Xq and half of the tile's rows
// of Wq in its shared memory; the leader's MMA warp drives both.  Warps 0 and 2
// load, warp 1 issues the MMAs, warps 4-11 (two per TMEM lane quarter, each
// half of the columns) dequantize and store.
template <GScale SC, OutKind KIND>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const float *__restrict__ x_scale, const float *__restrict__ w_scale,
                        const int32_t *__restrict__ offsets, uint8_t *__restrict__ y, int64_t ldy, int T, int E, int N,
                        int K, unsigned *err) {
  using L = PairTileSmem;
  constexpr bool kF8 = SC != GScale::I8, kBlock = SC == GScale::Block;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + L::kStages * L::kA;
  uint8_t *staging = smem + L::kRing;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + L::kStaging);
  uint64_t *empty = full + L::kStages;
  uint64_t *tfull = empty + L::kStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Groups g;
  g.row = reinterpret_cast<int *>(tmem_slot + 4);
  g.tile = g.row + kMaxExperts + 1;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = blockIdx.x / 2, units = gridDim.x / 2;
  const int ntn = (N + kPairCols - 1) / kPairCols;
  const int nk = (K + kBlk - 1) / kBlk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 2);  // the loaders of A and of B
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps * 2);  // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kPairCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncwarp();  // (thread 0 has just set up the barriers alone)
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();  // prologue done; the previous kernel's results are visible from here on
  pdl_trigger();
  build_groups(g, offsets, E, T, kPairRows, ntn);
  const int tiles = g.tile[E];

  if (warp < 4) regs_give();
  if (warp == 0 || warp == 2) {
    if (lane == 0) {
      // ---------------- TMA producers: warp 0 the rows of Xq, warp 2 those of Wq ----------------
      const bool x = warp == 0;
      const CUtensorMap *tm = x ? &tmA : &tmB;
      uint8_t *const ring = x ? sA : sB;
      const uint32_t bytes = x ? L::kA : L::kB;
      uint32_t stage = 0, phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      Place p;
      for (int tile = unit; tile < tiles && ok; tile += units) {
        p.find(g, E, tile, kPairRows);
        const int row = x ? p.row0 + p.mb * kPairRows + rank * 128
                          : p.e * N + p.nb * kPairCols + rank * (kPairCols / 2);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (leader) {  // its barrier counts both CTAs' copies
            mbar_arrive_expect_tx(&full[stage], 2 * bytes);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          tma_load_2d_pair(tm, mapa_shared(smem_u32(&full[stage]), 0), ring + stage * bytes, kb * kBlk, row);
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok && leader) {  // let every issued copy land before the CTA may exit
        for (int s = 0; s < L::kStages; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, nullptr, err);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer ----------------
      const int64_t mine = tiles > unit ? (tiles - unit + units - 1) / units : 0;  // this pair's tiles
      mma_loop<2, kF8, kBlock, L::kStages, 2, L::kA, L::kB, kPairCols>(
          smem_u32(sA), smem_u32(sB), full, empty, tfull, tempty, tmem_base, idesc8<kF8>(kPairRows, kPairCols),
          mine * nk, nk, nk, abort_flag, err);
      // every MMA issued above must finish before TMEM is released
      if (elect_one()) {
        umma_commit_pair(mapa_shared(smem_u32(drain), 0));
        mbar_wait(drain, 0, nullptr, err);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    regs_take();
    constexpr int kCols = kPairCols / 2;  // columns of this warp
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * kCols;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    auto release = [&](uint32_t b) {  // accumulator b may be overwritten, as far as this warp goes
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty0 + b * 8);
    };
    RowStore<KIND> out;
    out.stage = staging + (warp - 4) * kStageBytes;
    out.y = y;
    out.ldy = ldy;
    out.N = N;
    out.lane = lane;
    const int nbk = (N + kBlk - 1) / kBlk;
    uint32_t ab = 0, aphase = 0, stage = 0, phase = 0;
    bool ok = true;
    Place p;
    for (int tile = unit; tile < tiles && ok; tile += units) {
      p.find(g, E, tile, kPairRows);
      out.row0 = p.row0 + p.mb * kPairRows + rank * 128 + quarter * 32;
      out.row_end = p.row0 + p.rows;
      const int n0 = p.nb * kPairCols + half * kCols;
      const bool mine = out.row0 < out.row_end && n0 < N;  // uniform over the warp
      const int row = min(out.row0 + lane, T - 1);
      if constexpr (kBlock) {
        float2 acc[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
        const float *xs = x_scale + (int64_t)row * nk;
        const float *ws = w_scale + ((int64_t)p.e * nbk + min(n0 / kBlk, nbk - 1)) * nk;
        float s = __fmul_rn(__ldg(xs), __ldg(ws));
        // a block's product is complete when its operands are free again
        for (int kb = 0; kb < nk; ++kb) {
          const int kn = min(kb + 1, nk - 1);
          const float xn = __ldg(xs + kn), wn = __ldg(ws + kn);  // the next block's scales
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, abort_flag, err));
          if (!ok) break;
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
          tc_fence_after();
          const float2 s2 = make_float2(s, s);
          // columns 16 at a time: the next ones are on their way while these
          // are added up, and the accumulator is released before the last are
          uint32_t r[2][16];
          if (mine) {
            tmem_ld16(taddr + ab * kPairCols, r[0]);
            tmem_ld_wait();
          }
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            if (c + 1 == kCols / 16) {
              release(ab);
            } else if (mine) {
              tmem_ld16(taddr + ab * kPairCols + (c + 1) * 16, r[(c + 1) & 1]);
            }
            if (mine) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[c * 8 + j] = ffma2_rn(
                    make_float2(__uint_as_float(r[c & 1][2 * j]), __uint_as_float(r[c & 1][2 * j + 1])), s2,
                    acc[c * 8 + j]);
              if (c + 1 < kCols / 16) tmem_ld_wait();
            }
          }
          ab ^= 1;
          s = __fmul_rn(xn, wn);
        }
        if (ok && mine) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[2 * i] = acc[c * 16 + i].x;
              v[2 * i + 1] = acc[c * 16 + i].y;
            }
            out.put(v, n0 + c * 32);
          }
        }
      } else {
        const float dx = __ldg(x_scale + row);
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[ab], aphase, abort_flag, err));
        if (!ok) break;
        tc_fence_after();
        if (mine) {
#pragma unroll 1
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(taddr + ab * kPairCols + c * 32, r);
            tmem_ld_wait();
            float v[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int n = n0 + c * 32 + i * 4;
              const float4 dw = n < N ? __ldg(reinterpret_cast<const float4 *>(w_scale + (int64_t)p.e * N + n))
                                      : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              v[4 * i] = __fmul_rn(__fmul_rn(acc_value<kF8>(r[4 * i]), dx), dw.x);
              v[4 * i + 1] = __fmul_rn(__fmul_rn(acc_value<kF8>(r[4 * i + 1]), dx), dw.y);
              v[4 * i + 2] = __fmul_rn(__fmul_rn(acc_value<kF8>(r[4 * i + 2]), dx), dw.z);
              v[4 * i + 3] = __fmul_rn(__fmul_rn(acc_value<kF8>(r[4 * i + 3]), dx), dw.w);
            }
            out.put(v, n0 + c * 32);
          }
        }
        release(ab);
        ab ^= 1;
        if (ab == 0) aphase ^= 1;
      }
    }
  }

  __syncwarp();  // (of the loaders one lane has worked)
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's shared memory and TMEM stay live until the leader is done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kPairCols);
  }
}

// Clusters of `size` CTAs of a kernel (one CTA per SM) that `dev`, the current
// device, holds at once, after raising the kernel's shared-memory limit.
cudaError_t resident_clusters(const void *kern, int dev, int size, uint32_t smem, int *n) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && size == 1) {
    e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  } else if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(n, kern, &cfg);
  }
  if (e != cudaSuccess) cudaGetLastError();
  if (e == cudaErrorInvalidClusterSize) {  // a size that this device never runs
    *n = 0;
    e = cudaSuccess;
  }
  return e;
}

template <GScale SC, OutKind KIND>
cudaError_t pair_capacity(int dev, int *n) {
  static CapacityCache cache;
  const void *kern = reinterpret_cast<const void *>(grouped_pair_kernel<SC, KIND>);
  return cache.get(dev, n, [&](int *c) { return resident_clusters(kern, dev, 2, PairTileSmem::kTotal, c); });
}

template <GScale SC, OutKind KIND>
cudaError_t run_pair(const GroupedArgs &a, int cap, cudaStream_t st) {
  CUtensorMap tmA, tmB;
  if (!make_code_tmap(&tmA, a.xq, a.T, a.K, 128)) return cudaErrorInvalidValue;
  if (!make_code_tmap(&tmB, a.wq, a.E * a.N, a.K, kPairCols / 2)) return cudaErrorInvalidValue;
  // at most one tile more per group than its rows alone would need
  const int64_t groups = a.E < a.T ? a.E : a.T;
  const int64_t most = (a.T / kPairRows + groups) * ((a.N + kPairCols - 1) / kPairCols);
  const int units = (int)(most < cap ? most : cap);
  return launch_pdl(grouped_pair_kernel<SC, KIND>, dim3(units * 2), dim3(kThreads), PairTileSmem::kTotal, st, 2, tmA,
                    tmB, a.x_scale, a.w_scale, a.offsets, static_cast<uint8_t *>(a.y), a.ldy, (int)a.T, (int)a.E,
                    (int)a.N, (int)a.K, device_error_word());
}

// ---------------------------------------------------------------------------
// Small groups, and too few tiles to fill the SMs evenly: 128 x 128 tiles, one
// CTA each, whose K / 128 blocks are shared out too.  C clusters of S CTAs:
// cluster c owns the tiles c, c + C, ... and its CTAs share their (tile,
// block) items evenly, so a CTA holds the end of one tile, whole tiles, and
// the beginning of another.  Split tiles' partial sums meet in shared memory:
// every contributor adds up its share of the tile over all of them, in rank
// order, so results do not depend on timing.  No workspace, no atomics.  Of
// Xq's rows a box of 32, 64 or 128 is loaded, whichever holds what the group
// has: the MMA's other rows hold what the ring held before, and go nowhere.
// (One box a block: up to four of 32 rows cost the loader 730 cycles a block
// where one of 128 costs 545, 333 x 4096 x 11008: 34.9 -> 29.4 us.)
// ---------------------------------------------------------------------------
constexpr int kMaxSplit = 8;  // CTAs per cluster

// A split tile that this CTA helps to add up: cnt contributors from rank ra on
// (0: there is none), its expert, first row and first channel, and this CTA's
// share [u0, u1) of its units (four channels of a row, 32 units a row).
struct SplitTile {
  int cnt, ra, e, row, n, u0, u1;
};

struct SplitSmem {
  static constexpr uint32_t kA = 128 * kBlk;
  static constexpr uint32_t kB = 128 * kBlk;
  static constexpr int kStages = 5;
  static constexpr uint32_t kRing = kStages * (kA + kB);
  static constexpr uint32_t kStaging = kEpiWarps * kStageBytes;
  static constexpr uint32_t kTable = 2 * (kMaxExperts + 1) * 4 + 8;
  static constexpr int kBufs = 3;  // accumulators in flight; a fourth parks one
  static constexpr uint32_t kBars = (2 * kStages + 2 * kBufs + 1) * 8 + 16 + 2 * sizeof(SplitTile);
  static constexpr uint32_t kTotal = kRing + kStaging + kTable + kBars + 1024;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(2 * 128 * 128 * 4 <= kRing, "partial sums reuse the ring");
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <OutKind KIND>
__device__ __forceinline__ void put_four(uint8_t *y, int64_t i, const float (&v)[4]) {
  if constexpr (KIND == OutKind::F32) {
    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(y) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t p[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (KIND == OutKind::BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        p[k] = *reinterpret_cast<uint32_t *>(&h);
      } else {
        __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        p[k] = *reinterpret_cast<uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(y) + i) = make_uint2(p[0], p[1]);
  }
}

template <GScale SC, OutKind KIND>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA64,
                         const __grid_constant__ CUtensorMap tmA32, const __grid_constant__ CUtensorMap tmB,
                         const float *__restrict__ x_scale, const float *__restrict__ w_scale,
                         const int32_t *__restrict__ offsets, uint8_t *__restrict__ y, int64_t ldy, int T, int E, int N,
                         int K, FastDiv dS, FastDiv dC, FastDiv dnk, unsigned *err) {
  using L = SplitSmem;
  constexpr bool kF8 = SC != GScale::I8, kBlock = SC == GScale::Block;
  constexpr int kBufs = L::kBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sA = smem;
  uint8_t *sB = smem + L::kStages * L::kA;
  uint8_t *staging = smem + L::kRing;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + L::kStaging);
  uint64_t *empty = full + L::kStages;
  uint64_t *tfull = empty + L::kStages;
  uint64_t *tempty = tfull + kBufs;
  uint64_t *drain = tempty + kBufs;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  Groups g;
  g.row = reinterpret_cast<int *>(tmem_slot + 4);
  g.tile = g.row + kMaxExperts + 1;
  SplitTile *split = reinterpret_cast<SplitTile *>(g.tile + kMaxExperts + 1);  // [2]: slots 0 and 1

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int ntn = (N + 127) / 128, nk = dnk.d, S = dS.d, C = dC.d;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 2);  // the loaders of A and of B
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmA64);
    prefetch_tmap(&tmA32);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait();  // prologue done; the previous kernel's results are visible from here on
  pdl_trigger();
  build_groups(g, offsets, E, T, 128, ntn);

  // this cluster's tiles c, c + C, ...; this CTA's items [w0, w1) of theirs
  // (items * S < 2^31, see plan_split)
  const uint32_t c = dS.of(blockIdx.x), rank = blockIdx.x - c * S;
  const uint32_t items = dC.of(max(0, g.tile[E] - (int)c + C - 1)) * nk;
  const uint32_t w0 = dS.of(items * rank), w1 = dS.of(items * (rank + 1));

  if (warp == 0 || warp == 2) {
    if (lane == 0) {
      // ---------------- TMA producers: warp 0 the rows of Xq, warp 2 those of Wq ----------------
      const bool x = warp == 0;
      const uint64_t policy = policy_evict_first();
      uint32_t stage = 0, phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      Place p;
      for (uint32_t w = w0; w < w1 && ok;) {
        const uint32_t lt = dnk.of(w);
        int kb = w - lt * nk;
        const int kend = min(nk, (int)(w1 - lt * nk));
        p.find(g, E, c + lt * C, 128);
        const int row_a = p.row0 + p.mb * 128, row_b = p.e * N + p.nb * 128;
        // as many of the tile's rows as its group has: one box of 32, 64 or 128
        const int rows = p.rows - p.mb * 128, box = rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
        const CUtensorMap *const tm = !x ? &tmB : box == 32 ? &tmA32 : box == 64 ? &tmA64 : &tmA;
        const uint32_t bytes = x ? box * kBlk : L::kB;
        const int row = x ? row_a : row_b;
        // an expert's weights that one tile of rows reads once leave L2 first
        // (INT8, 192 rows of 64 experts 2048 -> 1408: 38.2 -> 36.9 us; of no
        // use to a dense weight)
        const bool once = !x && offsets != nullptr && p.rows <= 128;
        w += kend - kb;
        for (; kb < kend; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, err)) {
            ok = false;
            break;
          }
          uint8_t *const dst = x ? sA + stage * L::kA : sB + stage * L::kB;
          mbar_arrive_expect_tx(&full[stage], bytes);
          if (once) {
            tma_load_2d_hint(tm, &full[stage], dst, kb * kBlk, row, policy);
          } else {
            tma_load_2d(tm, &full[stage], dst, kb * kBlk, row);
          }
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {  // let every issued copy land before the CTA may exit
        for (int s = 0; s < L::kStages; ++s)
          if (armed & (1u << s)) mbar_wait(&full[s], (armed_parity >> s) & 1u, nullptr, err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    mma_loop<1, kF8, kBlock, L::kStages, kBufs, L::kA, L::kB, 128>(
        smem_u32(sA), smem_u32(sB), full, empty, tfull, tempty, tmem_base, idesc8<kF8>(128, 128), w1 - w0, nk,
        nk - (int)(w0 - dnk.of(w0) * nk), abort_flag, err);
    // every MMA issued above must finish before TMEM is released
    if (elect_one()) {
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr, err);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- the split tiles, worked out while the weights stream ----------------
    if (lane < 2) {
      const int slot = lane;
      SplitTile m{};
      if (S > 1 && w1 > w0) {
        const uint32_t lt = dnk.of(slot == 0 ? w0 : w1 - 1), i0 = lt * nk, i1 = i0 + nk;
        if (slot == 0 ? i0 < w0 : (i0 >= w0 && i1 > w1)) {
          // its contributors: the CTAs with its first to its last item
          m.ra = ((i0 + 1) * S - 1) / items;
          m.cnt = (i1 * S - 1) / items - m.ra + 1;
          Place p;
          p.find(g, E, c + lt * C, 128);
          m.e = p.e;
          m.row = p.row0 + p.mb * 128;
          m.n = p.nb * 128;
          const int units = min(128, p.rows - p.mb * 128) * 32;
          m.u0 = units * (rank - m.ra) / m.cnt;
          m.u1 = units * (rank - m.ra + 1) / m.cnt;
        }
      }
      split[slot] = m;
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: a row per lane, 64 columns per warp ----------------
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * 64;
    RowStore<KIND> out;
    out.stage = staging + (warp - 4) * kStageBytes;
    out.y = y;
    out.ldy = ldy;
    out.N = N;
    out.lane = lane;
    uint32_t ab = 0, aphase = 0, stage = 0, phase = 0;
    bool ok = true, parked = false, parked_row = false;
    // the last tile's sums go to slot 0 (begun by an earlier CTA) or to slot 1
    // (ended by a later one); worked out here, while the first block is loaded
    const uint32_t t0 = dnk.of(w0), t1 = w1 > w0 ? dnk.of(w1 - 1) : t0;
    const bool begun = w0 != t0 * nk && t0 == t1, ended = w1 == (t1 + 1) * nk;
    float2 acc[32];  // fp32 sums; for INT8 the bits of int32 sums
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = make_float2(0.0f, 0.0f);
    Place p;
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[ab]);
      if (++ab == kBufs) {
        ab = 0;
        aphase ^= 1;
      }
    };
    for (uint32_t w = w0; w < w1;) {
      const uint32_t lt = dnk.of(w);
      const int kb0 = w - lt * nk, kend = min(nk, (int)(w1 - lt * nk));
      p.find(g, E, c + lt * C, 128);
      out.row0 = p.row0 + p.mb * 128 + quarter * 32;
      out.row_end = p.row0 + p.rows;
      const int n0 = p.nb * 128 + half * 64;
      const bool mine = out.row0 < out.row_end && n0 < N;  // uniform over the warp
      const int row = min(out.row0 + lane, T - 1);
      w += kend - kb0;
      // this tile's scales, on their way while its blocks are multiplied
      const float dx = kBlock ? 0.0f : __ldg(x_scale + row);
      if (!kBlock && lane < 2 && n0 + lane * 32 < N) prefetch_l2(w_scale + (int64_t)p.e * N + n0 + lane * 32);
      if constexpr (kBlock) {
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = make_float2(0.0f, 0.0f);
        const float *xs = x_scale + (int64_t)row * nk;
        const float *ws = w_scale + ((int64_t)p.e * ntn + p.nb) * nk;
        float s = __fmul_rn(__ldg(xs + kb0), __ldg(ws + kb0));
        for (int kb = kb0; kb < kend; ++kb) {
          const int kn = min(kb + 1, nk - 1);
          const float xn = __ldg(xs + kn), wn = __ldg(ws + kn);  // the next block's scales
          // a block's product is complete when its operands are free again
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], phase, abort_flag, err));
          if (!ok) break;
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
          tc_fence_after();
          const float2 s2 = make_float2(s, s);
          const uint32_t src = taddr + ab * 128;
          // columns 16 at a time: the next ones are on their way while these
          // are added up, and the accumulator is released before the last are
          uint32_t r[2][16];
          if (mine) {
            tmem_ld16(src, r[0]);
            tmem_ld_wait();
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q == 3) {
              release();
            } else if (mine) {
              tmem_ld16(src + (q + 1) * 16, r[(q + 1) & 1]);
            }
            if (mine) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[q * 8 + j] = ffma2_rn(
                    make_float2(__uint_as_float(r[q & 1][2 * j]), __uint_as_float(r[q & 1][2 * j + 1])), s2,
                    acc[q * 8 + j]);
              if (q < 3) tmem_ld_wait();
            }
          }
          s = __fmul_rn(xn, wn);
        }
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&tfull[ab], aphase, abort_flag, err));
        if (ok) {
          tc_fence_after();
          if (mine) {
            uint32_t r[2][32];
            tmem_ld32(taddr + ab * 128, r[0]);
            tmem_ld32(taddr + ab * 128 + 32, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int h = j / 16, i = 2 * (j % 16);
              acc[j] = make_float2(__uint_as_float(r[h][i]), __uint_as_float(r[h][i + 1]));
            }
          }
          release();
        }
      }
      if (!ok) break;
      if (kb0 == 0 && kend == nk) {  // a whole tile
        if (mine) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              v[2 * j] = acc[h * 16 + j].x;
              v[2 * j + 1] = acc[h * 16 + j].y;
            }
            if constexpr (!kBlock) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int n = n0 + h * 32 + j * 4;
                const float4 dw = n < N ? __ldg(reinterpret_cast<const float4 *>(w_scale + (int64_t)p.e * N + n))
                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                v[4 * j] = __fmul_rn(__fmul_rn(acc_value<kF8>(__float_as_uint(v[4 * j])), dx), dw.x);
                v[4 * j + 1] = __fmul_rn(__fmul_rn(acc_value<kF8>(__float_as_uint(v[4 * j + 1])), dx), dw.y);
                v[4 * j + 2] = __fmul_rn(__fmul_rn(acc_value<kF8>(__float_as_uint(v[4 * j + 2])), dx), dw.z);
                v[4 * j + 3] = __fmul_rn(__fmul_rn(acc_value<kF8>(__float_as_uint(v[4 * j + 3])), dx), dw.w);
              }
            }
            out.put(v, n0 + h * 32);
          }
        }
      } else if (w < w1) {  // the end of a tile begun by an earlier CTA, with more to come: parked in TMEM
        parked = true;
        parked_row = out.row0 + lane < out.row_end;
        __syncwarp();  // (lane 0 has just released the accumulator alone; TMEM accesses take the whole warp)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t r[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            r[2 * j] = __float_as_uint(acc[q * 8 + j].x);
            r[2 * j + 1] = __float_as_uint(acc[q * 8 + j].y);
          }
          tmem_st16(taddr + kBufs * 128 + q * 16, r);
        }
        tmem_st_wait();
      }
    }
    if (S > 1 && ok) {
      // partial sums into the ring, which no load or MMA uses any more:
      // [slot][row of the tile][channel], slot 0 for a tile begun by an
      // earlier CTA, slot 1 for one that a later CTA ends; 16-byte chunks
      // swizzled by row; only the group's rows
      const int r = quarter * 32 + lane;
      uint4 *mine4 = reinterpret_cast<uint4 *>(smem) + r * 32;
      if (w1 > w0 && out.row0 + lane < out.row_end && (!ended || begun)) {
        uint4 *d = mine4 + (begun ? 0 : 128 * 32);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          d[(half * 16 + j) ^ (r & 7)] =
              make_uint4(__float_as_uint(acc[2 * j].x), __float_as_uint(acc[2 * j].y),
                         __float_as_uint(acc[2 * j + 1].x), __float_as_uint(acc[2 * j + 1].y));
      }
      if (parked) {
        // all of it before the stores, which some lanes make alone
        uint32_t v[4][16];
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld16(taddr + kBufs * 128 + q * 16, v[q]);
        tmem_ld_wait();
        if (parked_row) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t *four = v[j / 4] + 4 * (j % 4);
            mine4[(half * 16 + j) ^ (r & 7)] = make_uint4(four[0], four[1], four[2], four[3]);
          }
        }
      }
    }
  }

  __syncwarp();
  if (S > 1) {
    cluster_sync();  // every CTA's partial sums are written
#pragma unroll 1
    for (int slot = 0; slot < 2; ++slot) {
      const SplitTile m = split[slot];
      if (m.cnt == 0) continue;
      for (int u = m.u0 + threadIdx.x; u < m.u1; u += kThreads) {
        const int r = u >> 5, row = m.row + r, n = m.n + (u & 31) * 4;
        const uint32_t at = smem_u32(smem) + (uint32_t)(r * 32 + ((u & 31) ^ (r & 7))) * 16;
        if (n >= N) continue;
        float dx = 0.0f;
        float4 dw = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (!kBlock) {
          dx = __ldg(x_scale + row);
          dw = __ldg(reinterpret_cast<const float4 *>(w_scale + (int64_t)m.e * N + n));
        }
        uint32_t part[kMaxSplit][4];
#pragma unroll
        for (int q = 0; q < kMaxSplit; ++q)
          if (q < m.cnt) {  // the first contributor began the tile: its slot 1
            const uint4 v = ld_shared_cluster_v4(mapa_shared(at + (q == 0 ? 128 * 128 * 4 : 0), m.ra + q));
            part[q][0] = v.x;
            part[q][1] = v.y;
            part[q][2] = v.z;
            part[q][3] = v.w;
          }
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t sum = part[0][k];
#pragma unroll
          for (int q = 1; q < kMaxSplit; ++q)
            if (q < m.cnt) {
              if constexpr (kF8) {
                sum = __float_as_uint(__fadd_rn(__uint_as_float(sum), __uint_as_float(part[q][k])));
              } else {
                sum += part[q][k];
              }
            }
          v[k] = acc_value<kF8>(sum);
          if constexpr (!kBlock)
            v[k] = __fmul_rn(__fmul_rn(v[k], dx), k == 0 ? dw.x : k == 1 ? dw.y : k == 2 ? dw.z : dw.w);
        }
        put_four<KIND>(y, (int64_t)row * ldy + n, v);
      }
    }
    // no CTA leaves while a peer still reads its partial sums.  Nothing is
    // published, and what was read has been added up and stored, so the
    // barrier need not wait for the stores (1300 cycles of it)
    __syncwarp();
    cluster_sync_relaxed();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

template <GScale SC, OutKind KIND>
cudaError_t split_capacity(int dev, int S, int *n) {
  static CapacityCache cache[kMaxSplit + 1];
  const void *kern = reinterpret_cast<const void *>(grouped_split_kernel<SC, KIND>);
  return cache[S].get(dev, n, [&](int *c) { return resident_clusters(kern, dev, S, SplitSmem::kTotal, c); });
}

// How the split kernel is laid over the SMs: C clusters of S CTAs, and the
// blocks that the busiest CTA gets (cost).
struct SplitPlan {
  int S = 0, C = 0;
  int64_t cost = INT64_MAX;
};

// The split with the least cost.  One that splits tiles pays about 4 + S / 2
// blocks for its two cluster barriers and the partial sums (11008 x 4096 at
// one row: 14.1 us unsplit, 13.1 with S = 3, 12.9 with S = 6; 4096 x 4096 at
// one row: 12.1 us unsplit, 8.7, 7.8 and 7.1 with S = 2, 3 and 4, 8.7 with
// S = 8, of which fewer clusters fit).  Every CTA of a split cluster gets items
// (nk >= S), so that a tile's contributors are consecutive.  `tiles` is what the
// host reckons with, `most` what the offsets may lead to; tiles and a cluster's
// items are counted in 31 bits (beyond that, 10^16 operations, pairs have it).
template <GScale SC, OutKind KIND>
cudaError_t plan_split(int dev, int64_t tiles, int64_t most, int64_t nk, SplitPlan *plan) {
  SplitPlan best;
  for (int S = 1; S <= kMaxSplit && S <= nk; ++S) {
    int cap = 0;
    const cudaError_t e = split_capacity<SC, KIND>(dev, S, &cap);
    if (e != cudaSuccess) return e;
    const int64_t C = tiles < cap ? tiles : cap;
    if (C <= 0 || most > INT32_MAX / 2 || (most / C + 1) * nk * S >= INT32_MAX) continue;
    const int64_t cost = ((tiles + C - 1) / C * nk + S - 1) / S + (S > 1 ? 4 + S / 2 : 0);
    if (cost < best.cost) {
      best.S = S;
      best.C = (int)C;
      best.cost = cost;
    }
  }
  *plan = best;
  return cudaSuccess;
}

template <GScale SC, OutKind KIND>
cudaError_t run_split(const GroupedArgs &a, const SplitPlan &plan, cudaStream_t st) {
  CUtensorMap tmA, tmA64, tmA32, tmB;
  if (!make_code_tmap(&tmA32, a.xq, a.T, a.K, 32) || !make_code_tmap(&tmB, a.wq, a.E * a.N, a.K, 128))
    return cudaErrorInvalidValue;
  // (no tile has more rows than T: of T <= 32 and T <= 64 the larger maps stay unused)
  tmA = tmA64 = tmA32;
  if (a.T > 32 && !make_code_tmap(&tmA64, a.xq, a.T, a.K, 64)) return cudaErrorInvalidValue;
  if (a.T > 64 && !make_code_tmap(&tmA, a.xq, a.T, a.K, 128)) return cudaErrorInvalidValue;
  return launch_pdl(grouped_split_kernel<SC, KIND>, dim3(plan.C * plan.S), dim3(kThreads), SplitSmem::kTotal, st,
                    (unsigned)plan.S, tmA, tmA64, tmA32, tmB, a.x_scale, a.w_scale, a.offsets,
                    static_cast<uint8_t *>(a.y), a.ldy, (int)a.T, (int)a.E, (int)a.N, (int)a.K, FastDiv(plan.S),
                    FastDiv(plan.C), FastDiv((uint32_t)((a.K + kBlk - 1) / kBlk)), device_error_word());
}

// Row tiles of `rows` rows each over all groups.  The groups' sizes are on the
// device: the host reckons with rows spread evenly over as many groups as can
// have any, and half a tile of each group's last one empty.
int64_t row_tiles(const GroupedArgs &a, int64_t rows) {
  const int64_t groups = a.offsets == nullptr ? 1 : a.E < a.T ? a.E : a.T;
  if (groups <= 1) return (a.T + rows - 1) / rows;
  const int64_t spread = (2 * a.T + groups * rows) / (2 * rows);
  return spread > groups ? spread : groups;
}

// Pairs on 256 x 256 tiles or single CTAs on 128 x 128 ones: whichever's
// busiest unit has less to do.  A block of a pair's tile takes 1.35 times as
// long as one of a single's (block scales: 1.5 times, their sums waiting on
// both CTAs), for four times the products.  Singles and pairs, INT8: 12.5 and
// 15.1 us at 512 x 4096 x 4096, 20.1 and 16.2 at 1024 rows; 47.1 and 56.3 at
// 1100 x 4096 x 11008, whose 80 pairs' tiles do not fit at once; 4000 rows of
// 64 experts 2048 -> 1408, 35.4 and 46.8; 2000 of 8 4096 -> 4096, 52.6 and 42.6.
template <GScale SC, OutKind KIND>
cudaError_t run_grouped(const GroupedArgs &a, cudaStream_t st) {
  const int64_t nk = (a.K + kBlk - 1) / kBlk;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t ntn = (a.N + 127) / 128;
  SplitPlan split;
  e = plan_split<SC, KIND>(dev, row_tiles(a, 128) * ntn, (a.T / 128 + a.E) * ntn, nk, &split);
  if (e != cudaSuccess) return e;
  int cap = 0;
  e = pair_capacity<SC, KIND>(dev, &cap);
  if (e != cudaSuccess) return e;
  if (cap > 0) {
    const int64_t tiles = row_tiles(a, kPairRows) * ((a.N + kPairCols - 1) / kPairCols);
    const int64_t blocks = (tiles + cap - 1) / cap * nk;
    if (split.S == 0 || blocks * (SC == GScale::Block ? 30 : 27) < split.cost * 20)
      return run_pair<SC, KIND>(a, cap, st);
  }
  if (split.S == 0) return cudaErrorLaunchOutOfResources;
  return run_split<SC, KIND>(a, split, st);
}

template <GScale SC>
cudaError_t run_kind(const GroupedArgs &a, cudaStream_t st) {
  switch (a.kind) {
    case OutKind::F32: return run_grouped<SC, OutKind::F32>(a, st);
    case OutKind::F16: return run_grouped<SC, OutKind::F16>(a, st);
    default: return run_grouped<SC, OutKind::BF16>(a, st);
  }
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs &a, GScale scale, cudaStream_t st) {
  switch (scale) {
    case GScale::I8: return run_kind<GScale::I8>(a, st);
    case GScale::E4M3: return run_kind<GScale::E4M3>(a, st);
    default: return run_kind<GScale::Block>(a, st);
  }
}

}  // namespace sq
