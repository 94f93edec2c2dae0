// norm.hip -- residual addition, root-mean-square norm and MXFP8 quantize in
// one pass over the row (gfx950).
//
//   r = rnd(x + residual)                      (rnd: to the type of x; r = x without a residual)
//   y_i = r_i * w_i / sqrt(mean_j r_j^2 + eps)
//   (q, s) = MXFP8(y): blocks of 32, code max(expfield(amax) - 8, 0), E4M3 nearest even
//
// The norm is taken of the rounded r, the value that is stored and that the
// next layer adds to, so fused and unfused programs see the same stream.
//
// Roundings.  Squares, which fp64 holds exactly, are summed in fp64, and the
// row's factor is fp64, so neither leaves its range for finite rows (fp32 squares
// do from 1.8e19).  y is formed in fp32, which decides its E4M3 code unless the
// midpoint of two codes lies within 3 * 2^-23 of it; then, and where a block's
// largest |y| is that close to a power of two (its scale) or below 2^-64, or
// the factor below 2^-100, the wave's y are formed again in fp64 and rounded to
// odd, so that one rounding to the code remains.  (About 1 chunk of 64 lanes in
// 300 has such a lane.)
//
// Memory bound: x and residual are read once, r, q and s written once (7.03
// bytes an element in bf16); the row stays in registers between the sum and
// the quantize.
#include "mxq_device.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

// 8 consecutive elements as loaded, and as fp32.
template <bool kBf16>
struct Raw8 {
  u32x4 w[kBf16 ? 1 : 2];
};
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load_raw(const void* p, int64_t c) {
  constexpr int kN = kBf16 ? 1 : 2;
  Raw8<kBf16> r;
#pragma unroll
  for (int i = 0; i < kN; i++) r.w[i] = ((const u32x4*)p)[kN * c + i];
  return r;
}
// Streams (x, residual and r are touched once; times of variants in turn, in
// one graph's replays): in bf16 with the streaming hint (16384 x 8192: 168 ->
// 156 us; the codes are stored plainly, 161 with the hint).  An fp32 lane takes
// its 32 bytes in two instructions, and the hint makes those slower (8192 x
// 8192: 163 -> 181 us), so they are plain.
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load_raw_stream(const void* p, int64_t c) {
  if constexpr (!kBf16) return load_raw<kBf16>(p, c);
  return {__builtin_nontemporal_load((const u32x4*)p + c)};
}
template <bool kBf16>
__device__ __forceinline__ void to_f32(const Raw8<kBf16>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if constexpr (kBf16) v[i] = __uint_as_float(i & 1 ? r.w[0][i >> 1] & 0xFFFF0000u : r.w[0][i >> 1] << 16);
    else v[i] = __uint_as_float(r.w[i >> 2][i & 3]);
  }
}

// r again, as a value the compiler knows nothing of: it would keep the fp64
// values of the squares in registers for the branch of scale_quantize that
// seldom forms them again.
template <bool kBf16>
__device__ __forceinline__ void forget(Raw8<kBf16>& r) {
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); i++)
#pragma unroll
    for (int j = 0; j < 4; j++) asm volatile("" : "+v"(r.w[i][j]));
}

// a + b rounded to the stored type, in a.
template <bool kBf16>
__device__ __forceinline__ void add_round(Raw8<kBf16>& a, const Raw8<kBf16>& b) {
  float u[8], v[8];
  to_f32<kBf16>(a, u);
  to_f32<kBf16>(b, v);
#pragma unroll
  for (int i = 0; i < 8; i++) u[i] += v[i];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (kBf16) {
      a.w[0][i] = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)u[2 * i], (__bf16)u[2 * i + 1]});
    } else {
      a.w[0][i] = __float_as_uint(u[i]);
      a.w[1][i] = __float_as_uint(u[4 + i]);
    }
  }
}
template <bool kBf16>
__device__ __forceinline__ void store_raw_stream(void* p, int64_t c, const Raw8<kBf16>& r) {
  if constexpr (kBf16) {
    __builtin_nontemporal_store(r.w[0], (u32x4*)p + c);
  } else {
    ((u32x4*)p)[2 * c] = r.w[0];
    ((u32x4*)p)[2 * c + 1] = r.w[1];
  }
}

// v moved across lanes by a DPP control word (every lane reads a live one).
template <int kCtrl>
__device__ __forceinline__ double dpp64(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  const u32x2 moved = {(unsigned)__builtin_amdgcn_update_dpp(0, (int)w.x, kCtrl, 0xF, 0xF, false),
                       (unsigned)__builtin_amdgcn_update_dpp(0, (int)w.y, kCtrl, 0xF, 0xF, false)};
  return __builtin_bit_cast(double, moved);
}
__device__ __forceinline__ double lane64(double v, int lane) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, (u32x2){(unsigned)__builtin_amdgcn_readlane((int)w.x, lane),
                                            (unsigned)__builtin_amdgcn_readlane((int)w.y, lane)});
}
// Sum over the wave, in every lane: inside rows of 16 by DPP (lane ^ 1, lane ^
// 2, half row and row mirrored), then the four rows.
__device__ __forceinline__ double sum_wave(double v) {
  v += dpp64<kDppQuadXor1>(v);
  v += dpp64<kDppQuadXor2>(v);
  v += dpp64<0x141>(v);
  v += dpp64<0x140>(v);
  return (lane64(v, 0) + lane64(v, 16)) + (lane64(v, 32) + lane64(v, 48));
}

// Sum over the T threads of a row, the same in every thread and in every run
// (fixed tree).  part: one value per wave.
template <int T>
__device__ __forceinline__ double sum_row(double v, double* part) {
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

// In two chains, for their latency.
__device__ __forceinline__ double squares(const float (&v)[8]) {
  double s0 = 0, s1 = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    s0 = __builtin_fma((double)v[i], (double)v[i], s0);
    s1 = __builtin_fma((double)v[i + 1], (double)v[i + 1], s1);
  }
  return s0 + s1;
}

// 1 / sqrt(m), m = sum / k + eps: f within 2^-40, the fp32 reciprocal root and
// one Newton step in fp64 (1 x 8192 3.23 us, 3.29 with the library's root and
// divide), or in full where m leaves fp32's range.
struct Factor {
  double f, m;
};
__device__ __forceinline__ bool in_range(double m) { return m > 1e-30 && m < 1e30; }
__device__ __forceinline__ Factor row_factor(double sum, double inv_k, float eps) {
  const double m = sum * inv_k + (double)eps;
  if (!in_range(m)) return {1.0 / sqrt(m), m};
  const double y = (double)__builtin_amdgcn_rsqf((float)m);
  return {__builtin_fma(0.5 * y, __builtin_fma(-m * y, y, 1.0), y), m};
}
// f within 2^-50: one step more, where y is formed in fp64.
__device__ __forceinline__ double refined(const Factor& f) {
  return in_range(f.m) ? __builtin_fma(0.5 * f.f, __builtin_fma(-f.m * f.f, f.f, 1.0), f.f) : f.f;
}

// The MXFP8 block codes of y = r * f * w (see the top of the file): the codes
// of 1 - d and 1 + d times the fp32 y, d = 3 * 2^-23, are the same unless the
// midpoint of two codes, normal or subnormal, lies between them.  Three
// roundings put y within 3 * 2^-24 of its value, the two factors add 2^-24.
template <bool kBf16>
__device__ __forceinline__ u32x2 scale_quantize(Raw8<kBf16> r, Raw8<kBf16> weight, const Factor& factor,
                                                unsigned* code) {
  const float f32 = (float)factor.f;
  float v[8], w[8], y[8];
  to_f32<kBf16>(r, v);
  to_f32<kBf16>(weight, w);
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = v[i] * f32 * w[i];
  float big = 0;  // (in fp32: the instruction takes magnitudes of three; a NaN stays)
#pragma unroll
  for (int i = 0; i < 8; i++) big = __builtin_elementwise_maximum(big, __builtin_fabsf(y[i]));
  const unsigned top = quad_max(__float_as_uint(big)), c = e8m0_code_e4m3(top >> 23);
  // clamped to 8 units below 448 * 2^e, so that 1 + d times it is below that
  const float lim = __uint_as_float(mx8_limit_bits(c) - 8u);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float z = __builtin_amdgcn_fmed3f(y[i], -lim, lim);
    lo[i] = z * (1 - 0x3p-23f);
    hi[i] = z * (1 + 0x3p-23f);
  }
  const u32x2 out = mx8_convert8_f32(lo, c), other = mx8_convert8_f32(hi, c);
  *code = c;
  // (a factor or a largest this small: fp32 may have fewer bits than that)
  const bool again = ((out.x ^ other.x) | (out.y ^ other.y)) != 0 || f32 < 0x1p-100f ||
                     (top != 0 && (top < 0x1F800000u || ((top + 3u) & 0x7FFFFFu) <= 6u));
  if (__builtin_amdgcn_ballot_w64(again) == 0) return out;
  const double f = refined(factor);
  forget<kBf16>(r);
  forget<kBf16>(weight);
  to_f32<kBf16>(r, v);
  to_f32<kBf16>(weight, w);
#pragma unroll
  for (int i = 0; i < 8; i++) y[i] = round_odd((double)v[i] * f * (double)w[i]);
  return mx8_quantize_quad_f32(y, code);
}

// One row by T threads with U chunks of 8 elements each (k <= 8 T U): T = 64
// puts four rows into a block, one a wave.  Lanes of a chunk past k hold zeros
// and store nothing (skipping their waves measured slower where there are
// none); k % 32 == 0 keeps the quads of a block whole.  Measured (medians of a
// kernel trace): 16384 x 8192 bf16 with residual 148 us (6.4 TB/s), 8192 x 8192
// fp32 158, 1 x 8192 3.0.  The fp64 squares and the interval of y cost 2 % of the
// first and 0.2 us of the last (156 against 153 and 3.23 against 3.05 us in one
// graph's replays, fp32 even).
template <bool kBf16, bool kRes, int T, int U>
__global__ __launch_bounds__(T == 64 ? 256 : T) void k_rmsnorm_mx8(const void* x, const void* residual,
                                                                   const void* __restrict__ weight, int64_t rows,
                                                                   int64_t k, double inv_k, float eps, void* r,
                                                                   u32x2* __restrict__ q, uint8_t* __restrict__ s) {
  __shared__ double part[T / 64];
  const int tid = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = T == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  if (T == 64 && row >= rows) return;
  const int64_t lanes = k / 8, base = row * lanes;
  Raw8<kBf16> a[U], p[U], wr[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = u * T + tid;
    a[u] = {}, wr[u] = {};
    if (c >= lanes) continue;
    a[u] = load_raw_stream<kBf16>(x, base + c);
    if constexpr (kRes) p[u] = load_raw_stream<kBf16>(residual, base + c);
    wr[u] = load_raw<kBf16>(weight, c);
  }
  double sum = 0;
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = u * T + tid;
    if constexpr (kRes) {
      if (c < lanes) {
        add_round<kBf16>(a[u], p[u]);
        store_raw_stream<kBf16>(r, base + c, a[u]);
      }
    }
    float v[8];
    to_f32<kBf16>(a[u], v);
    sum += squares(v);
  }
  const Factor f = row_factor(sum_row<T>(sum, part), inv_k, eps);
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t c = u * T + tid;
    unsigned code;
    forget<kBf16>(a[u]);
    const u32x2 out = scale_quantize<kBf16>(a[u], wr[u], f, &code);
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
                                                           const void* __restrict__ weight, int64_t k, double inv_k,
                                                           float eps, void* r, u32x2* __restrict__ q,
                                                           uint8_t* __restrict__ s) {
  __shared__ double part[16];
  const int64_t lanes = k / 8, base = (int64_t)blockIdx.x * lanes;
  double sum = 0;
  for (int64_t c = threadIdx.x; c < lanes; c += 1024) {
    Raw8<kBf16> a = load_raw<kBf16>(x, base + c);
    if constexpr (kRes) {
      add_round<kBf16>(a, load_raw<kBf16>(residual, base + c));
      store_raw_stream<kBf16>(r, base + c, a);
    }
    float v[8];
    to_f32<kBf16>(a, v);
    sum += squares(v);
  }
  const Factor f = row_factor(sum_row<1024>(sum, part), inv_k, eps);
  for (int64_t c = threadIdx.x; c < lanes; c += 1024) {
    unsigned code;
    const u32x2 out = scale_quantize<kBf16>(load_raw<kBf16>(kRes ? r : x, base + c),  // what this thread itself stored
                                            load_raw<kBf16>(weight, c), f, &code);
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
                                     st>>>(x, residual, weight, rows, k, 1.0 / (double)k, eps, r, q2, s)
  // Without a residual a block of 512 has half the bytes on their way, and
  // twice the blocks of 256 do better once there are enough rows: 16384 x 8192
  // bf16 85 -> 77 us, 1024 rows even (8.4 and 8.5), 64 rows 3.5 us with 512
  // threads, 3.8 with 256.  (With a residual even, 156 and 155 us.)
  if constexpr (!kRes) {
    if (lanes > 512 && lanes <= 1024 && rows >= 1024) {
      MXQ_NORM(256, 4);
      return;
    }
  }
  if (lanes <= 64) MXQ_NORM(64, 1);
  else if (lanes <= 128) MXQ_NORM(64, 2);
  else if (lanes <= 256) MXQ_NORM(256, 1);
  else if (lanes <= 512) MXQ_NORM(256, 2);
  else if (lanes <= 1024) MXQ_NORM(512, 2);
  else if (lanes <= 2048) MXQ_NORM(1024, 2);
  else if (lanes <= 4096) MXQ_NORM(1024, 4);
  else
    k_rmsnorm_mx8_long<kBf16, kRes>
        <<<dim3((unsigned)rows), dim3(1024), 0, st>>>(x, residual, weight, k, 1.0 / (double)k, eps, r, q2, s);
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
