// sq_block.cu -- E4M3 quantizers with one scale per block of 128 (sm_100a).
//
//   activations  per token t and block b of 128 channels:
//                d_tb = max_{j in b} |x_tj inv_s_j| / 448,
//                code = e4m3(x_tj inv_s_j / d_tb)
//   weights      per 128 x 128 block of diag(s) W stored [N][K]:
//                d = max |s_j W_nj| / 448, code = e4m3(s_j W_nj / d)
//
// Both read every value once, hold a block in registers between its maximum
// and its codes, and write one byte per value: bound by HBM.
#include "sq_common.cuh"
#include "sq_internal.h"

namespace sq {

namespace {

constexpr int kBlk = 128;

// Codes of one vector of a block with scale delta.  FmtE4M3's reciprocal
// multiply needs fl(1 / delta) finite and accurate, so a block whose scale
// is below the normal range (absmax < 448 * 2^-126) divides every value.
template <int V>
__device__ __forceinline__ void block_codes(const float *v, float delta, float rcp, uint8_t *dst) {
  if (delta != 0.0f && delta < 0x1p-126f) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      w[i] = e4m3x2(__fdiv_rn(v[4 * i], delta), __fdiv_rn(v[4 * i + 1], delta)) |
             (e4m3x2(__fdiv_rn(v[4 * i + 2], delta), __fdiv_rn(v[4 * i + 3], delta)) << 16);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) reinterpret_cast<uint32_t *>(dst)[i] = w[i];
    return;
  }
  if constexpr (V == 8) {
    *reinterpret_cast<uint2 *>(dst) = FmtE4M3::codes8(v, delta, rcp);
  } else {
    *reinterpret_cast<uint32_t *>(dst) = FmtE4M3::codes4(v, delta, rcp);
  }
}

__device__ __forceinline__ float block_rcp(float delta) { return delta >= 0x1p-126f ? __frcp_rn(delta) : 0.0f; }

// Activations.  A warp owns a strip of kActUnroll * 32 vectors of 16 bytes
// (1024 channels at 16 bits, 512 at 32) and walks the rows with it, so its
// channels' inv_s stay in registers; a block of 128 channels is 16 lanes
// (16-bit values) or a whole warp (fp32) of one vector.
constexpr int kActUnroll = 4;
constexpr int kActWarps = 8;
template <typename T, bool kSmooth>
__global__ void __launch_bounds__(kActWarps * 32)
    quant_act_block_kernel(const T *__restrict__ x, int64_t rows, int64_t nvec, int64_t ld,
                           const float *__restrict__ inv_s, uint8_t *__restrict__ q, float *__restrict__ scale,
                           int64_t kb_count) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  constexpr int V = Vec<T>::N;
  constexpr int kLanes = kBlk / V;  // lanes of one block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t v0 = (int64_t)blockIdx.x * (kActUnroll * 32) + lane;
  const int64_t K = nvec * V;
  const uint64_t policy = policy_evict_first();  // every row is read exactly once
  float sc[kActUnroll][V];
  if constexpr (kSmooth) {
#pragma unroll
    for (int i = 0; i < kActUnroll; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) sc[i][e] = v0 + i * 32 < nvec ? __ldg(inv_s + (v0 + i * 32) * V + e) : 0.0f;
  }
  const int64_t step = (int64_t)gridDim.y * kActWarps;
  for (int64_t r = (int64_t)blockIdx.y * kActWarps + warp; r < rows; r += step) {
    uint4 raw[kActUnroll];
#pragma unroll
    for (int i = 0; i < kActUnroll; ++i)
      raw[i] = v0 + i * 32 < nvec ? ld_policy_v4(x + r * ld + (v0 + i * 32) * V, policy) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kActUnroll; ++i) {
      const int64_t v = v0 + i * 32;
      float f[V];
      Vec<T>::to_f32(raw[i], f);
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        if constexpr (kSmooth) {
          f[e] = __fmul_rn(f[e], sc[i][e]);
          f[e + 1] = __fmul_rn(f[e + 1], sc[i][e + 1]);
        }
        m = fmax3(m, fabsf(f[e]), fabsf(f[e + 1]));
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float delta = __fdiv_rn(m, 448.0f);
      if (v < nvec) {
        block_codes<V>(f, delta, block_rcp(delta), q + r * K + v * V);
        if ((lane & (kLanes - 1)) == 0) scale[r * kb_count + v / kLanes] = delta;
      }
    }
  }
}

// Weights: one CTA of 256 threads per 128 x 128 block, all of its vectors
// loaded before the first is used.  blockIdx.x: block column; blockIdx.y
// (and .z beyond 65535): block row over all experts, nb_count per expert.
constexpr int kWtThreads = 256;
template <typename T, bool kSmooth>
__global__ void __launch_bounds__(kWtThreads)
    quant_weight_block_kernel(const T *__restrict__ w, int64_t N, int64_t K, int64_t ld, int64_t nb_count,
                              int64_t block_rows, const float *__restrict__ s, uint8_t *__restrict__ q,
                              float *__restrict__ scale, int64_t kb_count) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  constexpr int V = Vec<T>::N;
  constexpr int kLanes = kBlk / V;               // threads across a block row
  constexpr int kRowsPass = kWtThreads / kLanes;  // block rows per pass
  constexpr int kPasses = kBlk / kRowsPass;
  __shared__ float red[32];
  const int64_t br = (int64_t)blockIdx.z * 65535 + blockIdx.y;
  if (br >= block_rows) return;
  const int64_t e = br / nb_count, nb = br % nb_count;
  const int64_t c = (int64_t)blockIdx.x * kBlk + (threadIdx.x % kLanes) * V;
  const int64_t n0 = nb * kBlk + threadIdx.x / kLanes;
  const T *we = w + e * N * ld;
  const uint64_t policy = policy_evict_first();
  uint4 raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = n0 + p * kRowsPass;
    raw[p] = c < K && n < N ? ld_policy_v4(we + n * ld + c, policy) : make_uint4(0, 0, 0, 0);
  }
  float sc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sc[i] = kSmooth && c < K ? __ldg(s + c + i) : 1.0f;
  float m = 0.0f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float f[V];
    Vec<T>::to_f32(raw[p], f);
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, fabsf(kSmooth ? __fmul_rn(f[i], sc[i]) : f[i]));
  }
  m = block_max(m, red);
  const float delta = __fdiv_rn(m, 448.0f), rcp = block_rcp(delta);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t n = n0 + p * kRowsPass;
    if (c < K && n < N) {
      float f[V];
      Vec<T>::to_f32(raw[p], f);
      if constexpr (kSmooth) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __fmul_rn(f[i], sc[i]);
      }
      block_codes<V>(f, delta, rcp, q + (e * N + n) * K + c);
    }
  }
  if (threadIdx.x == 0) scale[br * kb_count + blockIdx.x] = delta;
}

template <typename T>
cudaError_t act_block(const void *x, int64_t rows, int64_t cols, int64_t ld, const float *inv_s, uint8_t *q,
                      float *scale, cudaStream_t st) {
  constexpr int V = Vec<T>::N;
  const int64_t nvec = cols / V, strips = (nvec + kActUnroll * 32 - 1) / (kActUnroll * 32);
  // about eight CTAs per SM, so that each warp walks several rows
  int64_t gy = (rows + kActWarps - 1) / kActWarps;
  const int64_t most = ((int64_t)num_sms() * 8 + strips - 1) / strips;
  if (gy > most) gy = most;
  if (gy > 65535) gy = 65535;
  auto kern = inv_s != nullptr ? quant_act_block_kernel<T, true> : quant_act_block_kernel<T, false>;
  return launch_pdl(kern, dim3((unsigned)strips, (unsigned)gy), dim3(kActWarps * 32), 0, st, 1,
                    static_cast<const T *>(x), rows, nvec, ld, inv_s, q, scale, (cols + kBlk - 1) / kBlk);
}

template <typename T>
cudaError_t weight_block(const void *w, int64_t E, int64_t N, int64_t K, int64_t ld, const float *s, uint8_t *q,
                         float *scale, cudaStream_t st) {
  const int64_t nb = (N + kBlk - 1) / kBlk, kb = (K + kBlk - 1) / kBlk, rows = E * nb;
  const int64_t gz = (rows + 65534) / 65535, gy = rows < 65535 ? rows : 65535;
  if (gz > 65535) return cudaErrorNotSupported;
  auto kern = s != nullptr ? quant_weight_block_kernel<T, true> : quant_weight_block_kernel<T, false>;
  return launch_pdl(kern, dim3((unsigned)kb, (unsigned)gy, (unsigned)gz), dim3(kWtThreads), 0, st, 1,
                    static_cast<const T *>(w), N, K, ld, nb, rows, s, q, scale, kb);
}

}  // namespace

cudaError_t launch_quant_act_block(const void *x, sq_dtype xt, int64_t rows, int64_t cols, int64_t ld,
                                   const float *inv_s, uint8_t *q, float *scale, cudaStream_t st) {
  switch (xt) {
    case SQ_F32: return act_block<float>(x, rows, cols, ld, inv_s, q, scale, st);
    case SQ_F16: return act_block<__half>(x, rows, cols, ld, inv_s, q, scale, st);
    default: return act_block<__nv_bfloat16>(x, rows, cols, ld, inv_s, q, scale, st);
  }
}

cudaError_t launch_quant_weight_block(const void *w, sq_dtype wt, int64_t E, int64_t N, int64_t K, int64_t ld,
                                      const float *s, uint8_t *q, float *scale, cudaStream_t st) {
  switch (wt) {
    case SQ_F32: return weight_block<float>(w, E, N, K, ld, s, q, scale, st);
    case SQ_F16: return weight_block<__half>(w, E, N, K, ld, s, q, scale, st);
    default: return weight_block<__nv_bfloat16>(w, E, N, K, ld, s, q, scale, st);
  }
}

}  // namespace sq
