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
#include "sq_common.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kBlk = 128;          // channels per scale block = K bytes per stage
constexpr int kThreads = 384;      // TMA, MMA and two idle warps, then eight epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kStageBytes = 4096;  // an epilogue warp's output staging: 32 rows x 128 bytes

// Arrive on an mbarrier of another CTA of the cluster (shared::cluster
// address).  Without .release.cluster, which waits for the thread's earlier
// global stores: the TMEM reads that it publishes are ordered by
// tcgen05.wait::ld and the tcgen05 fences (per-block releases of the pair
// kernel, 4096 x 11008 x 4096: 365 -> 223 us).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Arrive once on the mbarrier at this address in both CTAs of the pair when
// the MMAs issued so far have completed.  One instruction for both: a commit
// holds the issuing thread for some 130 cycles, a quarter of a 128-channel
// block's MMAs.
__device__ __forceinline__ void umma_commit_both(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
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

// Where a tile lies.  find() is called with tile numbers that never fall.
struct Place {
  int e = 0, row0 = 0, rows = 0, mb = 0, nb = 0;
  __device__ __forceinline__ void find(const Groups &g, int tile, int tile_rows) {
    while (tile >= g.tile[e + 1]) ++e;
    row0 = g.row[e];
    rows = g.row[e + 1] - row0;
    const int nm = ceil_div_dev(rows, tile_rows), local = tile - g.tile[e];
    nb = local / nm;
    mb = local % nm;
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
  static constexpr int kCols = 128 / kEsz;  // columns per staged row
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

template <int CG, int BN>
struct GSmem {
  static constexpr int kStages = 5;
  static constexpr uint32_t kA = 128 * kBlk;        // this CTA's rows of Xq
  static constexpr uint32_t kB = (BN / CG) * kBlk;  // this CTA's share of the tile's rows of Wq
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

// Persistent over (128 CG) x BN tiles of Y, one CTA per SM.  CG = 2: a pair of
// CTAs works on one tile (tcgen05 cta_group::2), each with 128 rows of Xq and
// half of the tile's rows of Wq in its shared memory; the leader's MMA thread
// drives both.  Warp 0 loads, warp 1 issues the MMAs, warps 4-11 (two per
// TMEM lane quarter, each half of the columns) dequantize and store.
template <int CG, int BN, GScale SC, OutKind KIND>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const float *__restrict__ x_scale, const float *__restrict__ w_scale,
                        const int32_t *__restrict__ offsets, uint8_t *__restrict__ y, int64_t ldy, int T, int E, int N,
                        int K, unsigned *err) {
  using L = GSmem<CG, BN>;
  constexpr bool kF8 = SC != GScale::I8, kBlock = SC == GScale::Block;
  constexpr int kRows = 128 * CG;
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

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int unit = blockIdx.x / CG, units = gridDim.x / CG;
  const int ntn = (N + BN - 1) / BN;
  const int nk = (K + kBlk - 1) / kBlk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps * CG);  // the epilogue warps of every CTA on the tile
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_slot, 2 * BN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * BN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) {
    cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  } else {
    __syncthreads();
  }
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // prologue done; the previous kernel's results are visible from here on
  pdl_trigger();
  build_groups(g, offsets, E, T, kRows, ntn);
  const int tiles = g.tile[E];

  if (warp < 4) regs_give();
  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer ----------------
      uint32_t stage = 0, phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      Place p;
      for (int tile = unit; tile < tiles && ok; tile += units) {
        p.find(g, tile, kRows);
        const int row_a = p.row0 + p.mb * kRows + rank * 128, row_b = p.e * N + p.nb * BN + rank * (BN / CG);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (leader) {  // its barrier counts every CTA's copies
            mbar_arrive_expect_tx(&full[stage], CG * (L::kA + L::kB));
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          if constexpr (CG == 2) {
            const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
            tma_load_2d_pair(&tmA, bar, sA + stage * L::kA, kb * kBlk, row_a);
            tma_load_2d_pair(&tmB, bar, sB + stage * L::kB, kb * kBlk, row_b);
          } else {
            tma_load_2d(&tmA, &full[stage], sA + stage * L::kA, kb * kBlk, row_a);
            tma_load_2d(&tmB, &full[stage], sB + stage * L::kB, kb * kBlk, row_b);
          }
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
    if (lane == 0 && leader) {
      // ---------------- MMA issuer ----------------
      auto commit = [](uint64_t *bar) {
        if constexpr (CG == 2) {
          umma_commit_both(bar);
        } else {
          umma_commit(bar);
        }
      };
      constexpr uint32_t idesc = idesc8<kF8>(kRows, BN);
      uint32_t stage = 0, phase = 0, ab = 0, aphase = 0;
      bool ok = true;
      for (int tile = unit; tile < tiles && ok; tile += units) {
        for (int kb = 0; kb < nk; ++kb) {
          const bool first = kBlock || kb == 0, last = kBlock || kb == nk - 1;
          if (first && !mbar_wait(&tempty[ab], aphase ^ 1, abort_flag, err)) {
            ok = false;
            break;
          }
          if (!mbar_wait(&full[stage], phase, abort_flag, err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t a0 = desc_sw128_kmajor(smem_u32(sA + stage * L::kA));
          const uint64_t b0 = desc_sw128_kmajor(smem_u32(sB + stage * L::kB));
#pragma unroll
          for (int k = 0; k < kBlk / 32; ++k) {
            const uint32_t add = (k != 0 || !first) ? 1u : 0u;
            if constexpr (CG == 2) {
              umma8_pair<kF8>(tmem_base + ab * BN, a0 + 2 * k, b0 + 2 * k, idesc, add);
            } else {
              umma8<kF8>(tmem_base + ab * BN, a0 + 2 * k, b0 + 2 * k, idesc, add);
            }
          }
          commit(&empty[stage]);
          if (last) {
            if (!kBlock) commit(&tfull[ab]);
            ab ^= 1;
            if (ab == 0) aphase ^= 1;
          }
          if (++stage == L::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // every MMA issued above must finish before TMEM is released
      if constexpr (CG == 2) {
        umma_commit_pair(mapa_shared(smem_u32(drain), 0));
      } else {
        umma_commit(drain);
      }
      mbar_wait(drain, 0, nullptr, err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    regs_take();
    constexpr int kCols = BN / 2;  // columns of this warp
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + half * kCols;
    const uint32_t tempty0 = CG == 2 ? mapa_shared(smem_u32(tempty), 0) : 0u;
    auto release = [&](uint32_t b) {  // accumulator b may be overwritten, as far as this warp goes
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) {
          mbar_arrive_remote(tempty0 + b * 8);
        } else {
          mbar_arrive(&tempty[b]);
        }
      }
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
      p.find(g, tile, kRows);
      out.row0 = p.row0 + p.mb * kRows + rank * 128 + quarter * 32;
      out.row_end = p.row0 + p.rows;
      const int n0 = p.nb * BN + half * kCols;
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
            tmem_ld16(taddr + ab * BN, r[0]);
            tmem_ld_wait();
          }
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            if (c + 1 == kCols / 16) {
              release(ab);
            } else if (mine) {
              tmem_ld16(taddr + ab * BN + (c + 1) * 16, r[(c + 1) & 1]);
            }
            if (mine) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                acc[c * 8 + j] = ffma2_rn(make_float2(__uint_as_float(r[c & 1][2 * j]), __uint_as_float(r[c & 1][2 * j + 1])),
                                          s2, acc[c * 8 + j]);
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
            tmem_ld32(taddr + ab * BN + c * 32, r);
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

  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the peer's shared memory and TMEM stay live until the leader is done
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) {
      tmem_dealloc_pair(tmem_base, 2 * BN);
    } else {
      tmem_dealloc(tmem_base, 2 * BN);
    }
  }
}

// Sets the kernel's shared-memory limit once per device; the clusters of CG
// CTAs that can be resident at once (0: none, or a failed query).
template <int CG, int BN, GScale SC, OutKind KIND>
int gemm_capacity() {
  static int cache[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  int &c = cache[dev & 63];
  if (c == 0) {
    auto kern = grouped_gemm_kernel<CG, BN, SC, KIND>;
    constexpr uint32_t smem = GSmem<CG, BN>::kTotal;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
    if (CG == 1) {
      c = num_sms();
    } else {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(CG, 1, 1);
      cfg.blockDim = dim3(kThreads, 1, 1);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = CG;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return 0;
      c = n;
    }
  }
  return c;
}

template <int CG, int BN, GScale SC, OutKind KIND>
cudaError_t run_gemm(const GroupedArgs &a, cudaStream_t st) {
  constexpr int kRows = 128 * CG;
  CUtensorMap tmA, tmB;
  if (!make_code_tmap(&tmA, a.xq, a.T, a.K, 128)) return cudaErrorInvalidValue;
  if (!make_code_tmap(&tmB, a.wq, a.E * a.N, a.K, BN / CG)) return cudaErrorInvalidValue;
  const int cap = gemm_capacity<CG, BN, SC, KIND>();
  if (cap <= 0) return cudaErrorLaunchOutOfResources;
  // at most one tile more per group than its rows alone would need
  const int64_t groups = a.E < a.T ? a.E : a.T;
  const int64_t most = (a.T / kRows + groups) * ((a.N + BN - 1) / BN);
  const int units = (int)(most < cap ? most : cap);
  return launch_pdl(grouped_gemm_kernel<CG, BN, SC, KIND>, dim3(units * CG), dim3(kThreads), GSmem<CG, BN>::kTotal, st,
                    CG, tmA, tmB, a.x_scale, a.w_scale, a.offsets, static_cast<uint8_t *>(a.y), a.ldy, (int)a.T,
                    (int)a.E, (int)a.N, (int)a.K, device_error_word());
}

template <GScale SC, OutKind KIND>
cudaError_t run_grouped(const GroupedArgs &a, cudaStream_t st) {
  // pairs once 256 x 256 tiles occupy every pair and groups fill their rows
  const int64_t tiles = (a.T + 255) / 256 * ((a.N + 255) / 256);
  if (a.T / a.E >= 128 && tiles >= num_sms() / 2) return run_gemm<2, 256, SC, KIND>(a, st);
  return run_gemm<1, 128, SC, KIND>(a, st);
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
