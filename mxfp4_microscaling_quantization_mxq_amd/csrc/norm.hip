// norm.hip -- residual addition, root-mean-square norm and MXFP8 quantize in
// one pass over the row (gfx950).
//
//   r = rnd(x + residual)                      (rnd: to the type of x; r = x without a residual)
//   y_i = r_i * (1 / sqrt(mean_j r_j^2 + eps)) * w_i      (fp32, in this order)
//   (q, s) = MXFP8(y): blocks of 32, code max(expfield(amax) - 8, 0), E4M3 nearest even
//
// The norm is taken of the rounded r, the value that is stored and that the
// next layer adds to, so fused and unfused programs see the same stream.
// The sum of squares is held in fp32; mean, sum and square root of the row's
// one scale are in fp64 and rounded once, so every y_i carries two fp32
// roundings.
//
// Memory bound: x and residual are read once, r, q and s written once (7.03
// bytes an element in bf16); the row stays in registers between the sum and
// the quantize.
#include "mxq_device.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

// 8 consecutive elements (lane c of the row) as fp32.
template <bool kBf16>
__device__ __forceinline__ void load8_f32(const void* p, int64_t c, float (&v)[8]) {
  if constexpr (kBf16) {
    const u32x4 w = ((const u32x4*)p)[c];
    const unsigned ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = __uint_as_float(ww[i] << 16);
      v[2 * i + 1] = __uint_as_float(ww[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4 a = ((const f32x4*)p)[2 * c], b = ((const f32x4*)p)[2 * c + 1];
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
  }
}

// v rounded to the stored type; stores it at p unless p is null.
template <bool kBf16>
__device__ __forceinline__ void round_store8(void* p, int64_t c, float (&v)[8]) {
  if constexpr (kBf16) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const unsigned lo = f32_to_bf16_rne(v[2 * i]), hi = f32_to_bf16_rne(v[2 * i + 1]);
      w[i] = lo | (hi << 16);
      v[2 * i] = __uint_as_float(lo << 16);
      v[2 * i + 1] = __uint_as_float(hi << 16);
    }
    ((u32x4*)p)[c] = w;
  } else {
    ((f32x4*)p)[2 * c] = (f32x4){v[0], v[1], v[2], v[3]};
    ((f32x4*)p)[2 * c + 1] = (f32x4){v[4], v[5], v[6], v[7]};
  }
}

__device__ __forceinline__ float sum_wave(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Sum over the T threads of a row, the same in every thread and in every run
// (fixed tree).  part holds one float per wave of the block.
template <int T>
__device__ __forceinline__ float sum_row(float v, float* part) {
  v = sum_wave(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < T / 64; i++) v += part[i];
  }
  return v;
}

__device__ __forceinline__ float row_scale(float sum, int64_t k, float eps) {
  return (float)(1.0 / sqrt((double)sum / (double)k + (double)eps));
}

// One row by T threads with U chunks of 8 elements each (k <= 8 T U): T = 64
// puts four rows into a block, one a wave.  Lanes of a chunk past k hold
// zeros and store nothing; k % 32 == 0 keeps the quads of a block whole.
template <bool kBf16, bool kRes, int T, int U>
__global__ __launch_bounds__(T == 64 ? 256 : T) void k_rmsnorm_mx8(const void* x, const void* residual,
                                                                   const void* __restrict__ weight, int64_t rows,
                                                                   int64_t k, float eps, void* r,
                                                                   u32x2* __restrict__ q, uint8_t* __restrict__ s) {
  __shared__ float part[T / 64];
  const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = T == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (T == 64 && row >= rows) return;
  const int64_t lanes = k / 8, base = row * lanes;
  float v[U][8], w[U][8], sum = 0;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = u * T + tid;
#pragma unroll
    for (int i = 0; i < 8; i++) v[u][i] = 0, w[u][i] = 0;
    if (c >= lanes) continue;
    load8_f32<kBf16>(x, base + c, v[u]);
    load8_f32<kBf16>(weight, c, w[u]);
    if constexpr (kRes) {
      float p[8];
      load8_f32<kBf16>(residual, base + c, p);
#pragma unroll
      for (int i = 0; i < 8; i++) v[u][i] += p[i];
      round_store8<kBf16>(r, base + c, v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; u++)
#pragma unroll
    for (int i = 0; i < 8; i++) sum = __builtin_fmaf(v[u][i], v[u][i], sum);
  const float rs = row_scale(sum_row<T>(sum, part), k, eps);
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = u * T + tid;
#pragma unroll
    for (int i = 0; i < 8; i++) v[u][i] = v[u][i] * rs * w[u][i];
    unsigned code;
    const u32x2 out = mx8_quantize_quad_f32(v[u], &code);
    if (c < lanes) {
      q[base + c] = out;
      if ((c & 3) == 0) s[(base + c) >> 2] = (uint8_t)code;
    }
  }
}

// Rows longer than a block's registers hold: the second pass reads r (or x)
// again.
template <bool kBf16, bool kRes>
__global__ __launch_bounds__(1024) void k_rmsnorm_mx8_long(const void* x, const void* residual,
                                                           const void* __restrict__ weight, int64_t k, float eps,
                                                           void* r, u32x2* __restrict__ q, uint8_t* __restrict__ s) {
  __shared__ float part[16];
  const int64_t lanes = k / 8, base = (int64_t)blockIdx.x * lanes;
  float sum = 0;
  for (int64_t c = threadIdx.x; c < lanes; c += 1024) {
    float v[8];
    load8_f32<kBf16>(x, base + c, v);
    if constexpr (kRes) {
      float p[8];
      load8_f32<kBf16>(residual, base + c, p);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] += p[i];
      round_store8<kBf16>(r, base + c, v);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) sum = __builtin_fmaf(v[i], v[i], sum);
  }
  const float rs = row_scale(sum_row<1024>(sum, part), k, eps);
  for (int64_t c = threadIdx.x; c < lanes; c += 1024) {
    float v[8], w[8];
    load8_f32<kBf16>(kRes ? r : x, base + c, v);  // what this thread itself stored
    load8_f32<kBf16>(weight, c, w);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = v[i] * rs * w[i];
    unsigned code;
    const u32x2 out = mx8_quantize_quad_f32(v, &code);
    q[base + c] = out;
    if ((c & 3) == 0) s[(base + c) >> 2] = (uint8_t)code;
  }
}

template <bool kBf16, bool kRes>
void launch_norm(const void* x, const void* residual, const void* weight, int64_t rows, int64_t k, float eps, void* r,
                 uint8_t* q, uint8_t* s, hipStream_t st) {
  const int64_t lanes = k / 8;
  u32x2* q2 = (u32x2*)q;
#define MXQ_NORM(T, U)                                                                                             \
  k_rmsnorm_mx8<kBf16, kRes, T, U><<<dim3((unsigned)(T == 64 ? (rows + 3) / 4 : rows)), dim3(T == 64 ? 256 : T), 0, \
                                     st>>>(x, residual, weight, rows, k, eps, r, q2, s)
  if (lanes <= 64) MXQ_NORM(64, 1);
  else if (lanes <= 128) MXQ_NORM(64, 2);
  else if (lanes <= 256) MXQ_NORM(256, 1);
  else if (lanes <= 512) MXQ_NORM(256, 2);
  else if (lanes <= 1024) MXQ_NORM(256, 4);
  else if (lanes <= 2048) MXQ_NORM(1024, 2);
  else if (lanes <= 4096) MXQ_NORM(1024, 4);
  else
    k_rmsnorm_mx8_long<kBf16, kRes><<<dim3((unsigned)rows), dim3(1024), 0, st>>>(x, residual, weight, k, eps, r, q2, s);
#undef MXQ_NORM
}

}  // namespace

// Rows per launch: at most 2^31 threads.
constexpr int64_t kRowsPerLaunch = 1 << 21;

hipError_t launch_rmsnorm_quantize_fp8(const void* x, const void* residual, const void* weight, bool bf16,
                                       int64_t rows, int64_t k, float eps, void* r, uint8_t* q, uint8_t* s,
                                       hipStream_t st) {
  const int64_t e = bf16 ? 2 : 4;
  for (int64_t at = 0; at < rows; at += kRowsPerLaunch) {
    const int64_t n = std::min(kRowsPerLaunch, rows - at);
    const void* xt = (const uint8_t*)x + at * k * e;
    const void* pt = residual ? (const uint8_t*)residual + at * k * e : nullptr;
    void* rt = residual ? (uint8_t*)r + at * k * e : nullptr;
    uint8_t *qt = q + at * k, *stt = s + at * (k / 32);
    if (bf16)
      residual ? launch_norm<true, true>(xt, pt, weight, n, k, eps, rt, qt, stt, st)
               : launch_norm<true, false>(xt, pt, weight, n, k, eps, rt, qt, stt, st);
    else
      residual ? launch_norm<false, true>(xt, pt, weight, n, k, eps, rt, qt, stt, st)
               : launch_norm<false, false>(xt, pt, weight, n, k, eps, rt, qt, stt, st);
  }
  return hipGetLastError();
}

}  // namespace mxq
