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

// max(|a|, |b|, |c|) in one instruction (sm_100 three-input max).
__device__ __forceinline__ float fmax3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Codes of fl(v / delta) (IEEE division by the block's scale) without dividing
// every value, for scales of 2^-90 and more, rcp = fl(1 / delta):
//  1. lo = fl(rcp (1 - 2^-21)) and hi = fl(rcp (1 + 2^-21)): fl(v lo) and
//     fl(v hi) lie at least 2^-21 - 3 * 2^-24 of v / delta away from it, on
//     either side, and fl(v / delta) at most 2^-24 of it.  E4M3 rounding is
//     monotone, so equal codes at both ends are the code.
//  2. Where they differ, v / delta is next to a midpoint t of two E4M3 values
//     (values of few significant bits divided by each other often are: bf16
//     activations without smoothing, 16384 x 8192: 105 us with a division
//     here, 75 us).  q = fl(v rcp) is within 1.5 ulp of v / delta,
//     r = fl(v - delta q) and Q = q + r rcp exact but for r's and rcp's
//     rounding: within 1.5 * 2^-23 ulp.  fl(Q) and fl(v / delta) can only
//     have different codes with a float midpoint t +- ulp / 2 between them.
//     For t = k 2^i (16 <= k < 32) and delta = B 2^j (24-bit B), v - delta t is
//     an integer n times 2^(i + j), and it is delta ulp / 2 = B 2^-20 of these
//     units to within B 2^-41: so B is within 16 of a multiple of 2^20 (and not
//     that multiple, which no 24-bit v reaches).
//  3. Such a delta's values, and those of smaller scales, are divided.
// An all-zero block, and one whose scale underflows to 0, has codes +0.
struct BlockScale {
  float delta, rcp;
  float2 lo, hi;
  int step;  // how far down this list a value may have to go
};

__device__ __forceinline__ BlockScale block_scale(float absmax) {
  BlockScale s;
  // (kept off the division's slow path, which zero blocks would take too)
  s.delta = __fdiv_rn(fmaxf(absmax, 0x1p-80f), 448.0f);
  if (absmax < 0x1p-80f) s.delta = absmax == 0.0f ? 0.0f : __fdiv_rn(absmax, 448.0f);
  s.rcp = __frcp_rn(fmaxf(s.delta, 0x1p-90f));
  const float l = __fmul_rn(s.rcp, 1.0f - 0x1p-21f), h = __fmul_rn(s.rcp, 1.0f + 0x1p-21f);
  s.lo = make_float2(l, l);
  s.hi = make_float2(h, h);
  const uint32_t bits = __float_as_uint(s.delta);
  s.step = s.delta < 0x1p-90f ? 3 : ((bits + 16u) & 0xfffffu) <= 32u && (bits & 0xfffffu) != 0u ? 2 : 1;
  return s;
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) { return e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16); }

// fl(v + (v - delta q) rcp) of step 2, with v's sign where it is a zero
__device__ __forceinline__ float2 quotients(float2 v, float delta, float rcp) {
  const float2 y = make_float2(rcp, rcp), q = fmul2_rn(v, y);
  const float2 z = ffma2_rn(ffma2_rn(make_float2(-delta, -delta), q, v), y, q);
  return make_float2(copysignf(z.x, v.x), copysignf(z.y, v.y));
}

__device__ __noinline__ uint32_t codes_divided(float2 a, float2 b, float delta) {
  return e4m3x4(make_float2(__fdiv_rn(a.x, delta), __fdiv_rn(a.y, delta)),
                make_float2(__fdiv_rn(b.x, delta), __fdiv_rn(b.y, delta)));
}

// Four codes of a block.
__device__ __forceinline__ uint32_t block_codes4(float2 a, float2 b, const BlockScale &s) {
  const uint32_t w = e4m3x4(fmul2_rn(a, s.lo), fmul2_rn(b, s.lo));
  const uint32_t h = e4m3x4(fmul2_rn(a, s.hi), fmul2_rn(b, s.hi));
  if (w == h && s.step < 3) return w;
  if (s.step == 1) return e4m3x4(quotients(a, s.delta, s.rcp), quotients(b, s.delta, s.rcp));
  return s.delta == 0.0f ? 0u : codes_divided(a, b, s.delta);
}

// One 16-byte vector as fp32 pairs, times the channels' factors.
template <typename T, bool kScaled>
__device__ __forceinline__ void load_pairs(const uint4 &raw, const float2 *factor, float2 (&v)[Vec<T>::N / 2]) {
  float f[Vec<T>::N];
  Vec<T>::to_f32(raw, f);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) {
    v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    if constexpr (kScaled) v[i] = fmul2_rn(v[i], factor[i]);
  }
}

template <int P>
__device__ __forceinline__ float absmax_pairs(const float2 (&v)[P], float m) {
#pragma unroll
  for (int i = 0; i < P; ++i) m = fmax3_abs(m, v[i].x, v[i].y);
  return m;
}

template <int P>
__device__ __forceinline__ void store_codes(const float2 (&v)[P], const BlockScale &s, uint8_t *dst, bool store) {
  if constexpr (P == 4) {
    const uint2 w = make_uint2(block_codes4(v[0], v[1], s), block_codes4(v[2], v[3], s));
    if (store) *reinterpret_cast<uint2 *>(dst) = w;
  } else {
    const uint32_t w = block_codes4(v[0], v[1], s);
    if (store) *reinterpret_cast<uint32_t *>(dst) = w;
  }
}

// Activations.  A group of lanes holds one block, kActVecs 16-byte vectors
// per lane (4 lanes at 16 bits, 8 at 32), so that the shuffles, the division
// and the reciprocal of a block's scale are shared by 32 values (16 at 32
// bits): with one vector per lane the kernel was bound by instructions, 24 per
// value (16384 x 8192 bf16: 117 us, 3.5 TB/s).  The grid's groups cover
// row_step whole rows; a group walks down the rows from its block to the one
// row_step below, so its channels' inv_s stay in registers, the next row's
// vectors on their way.
constexpr int kActVecs = 4;
constexpr int kActWarps = 4;
constexpr int kActCtas = 4;  // per SM: 16 warps at up to 128 registers
template <typename T, bool kSmooth>
__global__ void __launch_bounds__(kActWarps * 32, kActCtas)
    quant_act_block_kernel(const T *__restrict__ x, int64_t rows, int64_t nvec, int64_t ld,
                           const float *__restrict__ inv_s, uint8_t *__restrict__ q, float *__restrict__ scale,
                           int64_t kb_count, int64_t row_step) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  constexpr int V = Vec<T>::N, P = V / 2;
  constexpr int kLanes = kBlk / (V * kActVecs);  // lanes of one block
  const int64_t group = ((int64_t)blockIdx.x * (kActWarps * 32) + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  int64_t r = group / kb_count;
  const int64_t kb = group % kb_count;
  const bool mine = r < row_step;
  const int64_t v0 = kb * (kBlk / V) + l;        // this lane's vectors: v0 + i * kLanes
  const uint64_t policy = policy_evict_first();  // every row is read exactly once
  float2 sc[kActVecs][P];
  if constexpr (kSmooth) {
#pragma unroll
    for (int i = 0; i < kActVecs; ++i)
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int64_t v = v0 + i * kLanes;
        sc[i][e] = v < nvec ? __ldg(reinterpret_cast<const float2 *>(inv_s + v * V) + e) : make_float2(0.0f, 0.0f);
      }
  }
  const T *src = x + r * ld + v0 * V;
  uint8_t *dst = q + r * (nvec * V) + v0 * V;
  uint4 raw[kActVecs];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < kActVecs; ++i)
      raw[i] = mine && row < rows && v0 + i * kLanes < nvec ? ld_policy_v4(src + i * kLanes * V, policy)
                                                            : make_uint4(0, 0, 0, 0);
  };
  fetch(r);
  // (the same number of passes for every group of a warp: they shuffle)
  for (int64_t left = (rows + row_step - 1) / row_step; left > 0; --left) {
    float2 f[kActVecs][P];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kActVecs; ++i) {
      load_pairs<T, kSmooth>(raw[i], sc[i], f[i]);
      m = absmax_pairs(f[i], m);
    }
    src += row_step * ld;
    fetch(r + row_step);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = block_scale(m);
    const bool store = mine && r < rows;
#pragma unroll
    for (int i = 0; i < kActVecs; ++i) store_codes(f[i], s, dst + i * kLanes * V, store && v0 + i * kLanes < nvec);
    if (store && l == 0) scale[r * kb_count + kb] = s.delta;
    r += row_step;
    dst += row_step * (nvec * V);
  }
}

// Weights: one CTA of 256 threads per 128 x 128 block, all of its vectors
// loaded before the first is used.  blockIdx.x: block column; blockIdx.y
// (and .z beyond 65535): block row over all experts, nb_count per expert.
constexpr int kWtThreads = 256;
template <typename T, bool kSmooth>
__global__ void __launch_bounds__(kWtThreads, sizeof(T) == 2 ? 3 : 2)
    quant_weight_block_kernel(const T *__restrict__ w, int64_t N, int64_t K, int64_t ld, int64_t nb_count,
                              int64_t block_rows, const float *__restrict__ s, uint8_t *__restrict__ q,
                              float *__restrict__ scale, int64_t kb_count) {
  pdl_wait();  // the previous kernel's results are visible from here on
  pdl_trigger();
  constexpr int V = Vec<T>::N, P = V / 2;
  constexpr int kLanes = kBlk / V;                // threads across a block row
  constexpr int kRowsPass = kWtThreads / kLanes;  // block rows per pass
  constexpr int kPasses = kBlk / kRowsPass;
  __shared__ float red[32];
  const int64_t br = (int64_t)blockIdx.z * 65535 + blockIdx.y;
  if (br >= block_rows) return;
  const int64_t e = br / nb_count, n0 = (br % nb_count) * kBlk + threadIdx.x / kLanes;
  const int64_t c = (int64_t)blockIdx.x * kBlk + (threadIdx.x % kLanes) * V;
  // rows of this thread's passes inside the matrix: n0 + p * kRowsPass < N
  const int passes = c < K ? (int)min((int64_t)kPasses, (N - n0 + kRowsPass - 1) / kRowsPass) : 0;
  const uint64_t policy = policy_evict_first();
  const T *src = w + (e * N + n0) * ld + c;
  uint4 raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    raw[p] = p < passes ? ld_policy_v4(src, policy) : make_uint4(0, 0, 0, 0);
    src += kRowsPass * ld;
  }
  float2 sc[P];
  if constexpr (kSmooth) {
#pragma unroll
    for (int i = 0; i < P; ++i)
      sc[i] = c < K ? __ldg(reinterpret_cast<const float2 *>(s + c) + i) : make_float2(0.0f, 0.0f);
  }
  float m = 0.0f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float2 f[P];
    load_pairs<T, kSmooth>(raw[p], sc, f);
    m = absmax_pairs(f, m);
  }
  m = block_max(m, red);
  const BlockScale bs = block_scale(m);
  uint8_t *dst = q + (e * N + n0) * K + c;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float2 f[P];
    load_pairs<T, kSmooth>(raw[p], sc, f);
    store_codes(f, bs, dst, p < passes);
    dst += kRowsPass * K;
  }
  if (threadIdx.x == 0) scale[br * kb_count + blockIdx.x] = bs.delta;
}

template <typename T>
cudaError_t act_block(const void *x, int64_t rows, int64_t cols, int64_t ld, const float *inv_s, uint8_t *q,
                      float *scale, cudaStream_t st) {
  constexpr int V = Vec<T>::N, kGroups = kActWarps * 32 * V * kActVecs / kBlk;  // groups per CTA
  const int64_t kb = (cols + kBlk - 1) / kBlk;
  // whole rows that the resident groups cover, evened out over the passes
  int64_t step = (int64_t)num_sms() * kActCtas * kGroups / kb;
  if (step < 1) step = 1;
  const int64_t passes = (rows + step - 1) / step;
  step = (rows + passes - 1) / passes;
  auto kern = inv_s != nullptr ? quant_act_block_kernel<T, true> : quant_act_block_kernel<T, false>;
  return launch_pdl(kern, dim3((unsigned)((step * kb + kGroups - 1) / kGroups)), dim3(kActWarps * 32), 0, st, 1,
                    static_cast<const T *>(x), rows, cols / V, ld, inv_s, q, scale, kb, step);
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
