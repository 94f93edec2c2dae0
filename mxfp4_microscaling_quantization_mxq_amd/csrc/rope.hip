// rope.hip -- rotation of new queries and keys by their positions, with the
// write of keys and values into the paged MXFP8 / MXFP4 cache (gfx950).
//
//   (a, b) -> (a cos - b sin, b cos + a sin),  angle = position * freqs[i]
//
// for pair i of a head's first 2 n elements, (i, n + i) or (2 i, 2 i + 1).  Keys
// are quantized from the rotated values as they are (no rounding to 16 bits
// between), values as they come.
//
// Roundings.  The angle is the product of the position (all 64 bits) and the fp32
// frequency in two fp64 terms, within 2^-66, reduced by pi / 2 in fp64, so far
// positions turn as exactly as near ones; cos and sin are fp64, within 2^-50.
// Keys are turned in fp64 and rounded to odd in fp32, so the one rounding to a
// code that follows is that of the fp64 value.  Queries, whose output is bf16, are
// turned in fp32 (three roundings of 2^-24).
//
// Memory bound: q, k and v are read once, q's bf16 and the codes written once
// (64 query heads over 8, D = 128, bf16 in, MXFP8: 39 kB a token).  16384 such
// tokens take 144 us, 4.4 TB/s (a copy of 4 GiB reaches 4.8), 2048 take 22 and one
// takes 3.6, of which a launch is about 3.
#include "mxq_device.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = kThreads * 8 / 2;  // pairs of a block's tokens: one for two elements of its lanes

struct RopeParams {
  RopeArgs a;
  KvShape c;
  unsigned lanes, rows;         // lanes of 8 elements a head; heads that a block's threads hold at a time
  unsigned tokens, heads_each;  // tokens of a block, and the heads it takes
};

// cos and sin of position * freq.  The position is p + rest (rest is 0 below 2^53).
// n is the nearest multiple of pi / 2 (two fp64 terms, 107 bits), the angle less
// that is in [-pi / 4, pi / 4] up to a rounding of n, where the Taylor polynomials
// end below 2^-54 (the sine's next term is r^17 / 17!).  Angles of 2^40 and more give NaN.
__device__ __forceinline__ double2 cos_sin(int64_t position, double freq) {
  const double high = (double)(int)(position >> 32) * 0x1p32, low = (double)(unsigned)position;
  const double p = high + low, rest = low - (p - high);
  const double hi = p * freq, lo = __builtin_fma(rest, freq, __builtin_fma(p, freq, -hi));
  const double n = __builtin_rint(hi * 0x1.45f306dc9c883p-1);
  const double r = __builtin_fma(-n, 0x1.1a62633145c07p-54, __builtin_fma(-n, 0x1.921fb54442d18p+0, hi)) + lo;
  const double z = r * r;
  double s = -1.0 / 1307674368000.0, c = 1.0 / 20922789888000.0;
  s = __builtin_fma(s, z, 1.0 / 6227020800.0), c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0), c = __builtin_fma(c, z, 1.0 / 479001600.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0), c = __builtin_fma(c, z, -1.0 / 3628800.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0), c = __builtin_fma(c, z, 1.0 / 40320.0);
  s = __builtin_fma(s, z, 1.0 / 120.0), c = __builtin_fma(c, z, -1.0 / 720.0);
  s = __builtin_fma(s, z, -1.0 / 6.0), c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  s = __builtin_fma(s * z, r, r), c = __builtin_fma(c, z, 1.0);
  const int quarter = (int)(n - 4.0 * __builtin_floor(0.25 * n));
  double2 o = {quarter & 1 ? s : c, quarter & 1 ? c : s};
  if (quarter == 1 || quarter == 2) o.x = -o.x;
  if (quarter & 2) o.y = -o.y;
  if (!(__builtin_fabs(hi) < 0x1p40)) o.x = o.y = __builtin_nan("");
  return o;
}

// 8 consecutive elements as loaded.
template <bool kBf16>
struct Eight {
  u32x4 w[kBf16 ? 1 : 2];
};
template <bool kBf16>
__device__ __forceinline__ Eight<kBf16> load8(const void* p, int64_t element) {
  Eight<kBf16> r;
  const u32x4* w = (const u32x4*)((const uint8_t*)p + element * (kBf16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); i++) r.w[i] = w[i];
  return r;
}
template <bool kBf16>
__device__ __forceinline__ float at8(const Eight<kBf16>& r, int i) {
  if constexpr (kBf16) return __uint_as_float(i & 1 ? r.w[0][i >> 1] & 0xFFFF0000u : r.w[0][i >> 1] << 16);
  else return __uint_as_float(r.w[i >> 2][i & 3]);
}

// A block takes `tokens` tokens and a run of heads (query heads, then key heads,
// then value heads): first the cos and sin of its tokens' pairs, into LDS, then
// head after head.  A lane keeps its token and its 8 elements of the head, so
// its factors stay in registers; four lanes are one block of the cache's formats.
template <bool kBf16, bool kFp4, bool kInter>
__global__ __launch_bounds__(kThreads) void k_rope_append(RopeParams p) {
  __shared__ double2 table[kTable];
  const RopeArgs& a = p.a;
  const unsigned n = a.pairs;
  const unsigned splits = (a.q_heads + 2 * p.c.heads + p.heads_each - 1) / p.heads_each;
  const int64_t t0 = (int64_t)(blockIdx.x / splits) * p.tokens;
  const unsigned h0 = blockIdx.x % splits * p.heads_each;
  const unsigned here = (unsigned)min((int64_t)p.tokens, a.tokens - t0);
  for (unsigned i = threadIdx.x; i < here * n; i += kThreads) {
    const unsigned t = i / n, pair = i % n;
    const int64_t axis = a.axes ? min((int64_t)a.axes[pair], a.position_axes - 1) : 0;
    table[i] = cos_sin(a.positions[axis * a.tokens + t0 + t], (double)a.freqs[pair]);
  }
  __syncthreads();

  const unsigned row = threadIdx.x / p.lanes, e8 = threadIdx.x % p.lanes;
  const unsigned t = row % p.tokens, sub = row / p.tokens, step = p.rows / p.tokens;
  if (sub >= step || t >= here) return;
  const int64_t token = t0 + t, slot = a.slots[token];
  const bool kept = slot >= 0 && slot < p.c.pages << p.c.page_shift;
  // this lane's pairs: turned with the elements `other` further on, by -sin in
  // the first half of the pairs and +sin in the second
  const unsigned first = 8 * e8;
  const bool turned = first < 2 * n, second = !kInter && first >= n;
  const int other = kInter || !turned ? 0 : second ? -(int)n : (int)n;
  const double2* mine = table + t * n + (kInter ? first / 2 : second ? first - n : first);
  float co[kInter ? 4 : 8], si[kInter ? 4 : 8];
#pragma unroll
  for (int i = 0; i < (kInter ? 4 : 8); i++) {
    const double2 f = turned ? mine[i] : (double2){1, 0};
    co[i] = (float)f.x, si[i] = second ? (float)f.y : -(float)f.y;
  }

  const unsigned all = a.q_heads + 2 * p.c.heads, h1 = min(h0 + p.heads_each, all);
  for (unsigned h = h0 + sub; h < h1; h += step) {
    const bool query = h < a.q_heads, value = h >= a.q_heads + p.c.heads;
    const unsigned head = query ? h : value ? h - a.q_heads - p.c.heads : h - a.q_heads;
    const void* src = query ? a.q : value ? a.v : a.k;
    const int64_t from = token * (query ? a.q_stride : value ? a.v_stride : a.k_stride) + (int64_t)head * p.c.dim + first;
    if (query) {
      const Eight<kBf16> x = load8<kBf16>(src, from), y = load8<kBf16>(src, from + other);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if constexpr (kInter) {
          const float u = at8<kBf16>(x, i), w = at8<kBf16>(x, i ^ 1);
          o[i] = __builtin_fmaf(u, co[i / 2], w * (i & 1 ? -si[i / 2] : si[i / 2]));
        } else {
          o[i] = __builtin_fmaf(at8<kBf16>(x, i), co[i], at8<kBf16>(y, i) * si[i]);
        }
        if (!turned) o[i] = at8<kBf16>(x, i);
      }
      u32x4 out;
#pragma unroll
      for (int i = 0; i < 4; i++) out[i] = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)o[2 * i], (__bf16)o[2 * i + 1]});
      *(u32x4*)(a.q_out + (token * a.q_heads + head) * p.c.dim + first) = out;
      continue;
    }
    if (!kept) continue;
    const Eight<kBf16> x = load8<kBf16>(src, from);
    unsigned code;
    u32x2 out;
    if (value) {
      if constexpr (kBf16) {
        const bf16x8 xb = __builtin_bit_cast(bf16x8, x.w[0]);
        if constexpr (kFp4) out.x = mx_quantize_quad_bf16(xb, &code);
        else out = mx8_quantize_quad_bf16(xb, &code);
      } else {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; i++) o[i] = at8<kBf16>(x, i);
        if constexpr (kFp4) out.x = mx_quantize_quad_f32(o, &code);
        else out = mx8_quantize_quad_f32(o, &code);
      }
    } else {
      const Eight<kBf16> y = load8<kBf16>(src, from + other);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        o[i] = at8<kBf16>(x, i);
        if (!turned) continue;
        const double2 f = mine[kInter ? i / 2 : i];
        const double w = at8<kBf16>(kInter ? x : y, kInter ? i ^ 1 : i);
        const bool plus = kInter ? (i & 1) != 0 : second;
        o[i] = round_odd(__builtin_fma((double)o[i], f.x, w * (plus ? f.y : -f.y)));
      }
      if constexpr (kFp4) out.x = mx_quantize_quad_f32(o, &code);
      else out = mx8_quantize_quad_f32(o, &code);
    }
    const int64_t ph = (slot >> p.c.page_shift) * p.c.heads + head;
    const int64_t pos = slot & ((1 << p.c.page_shift) - 1);
    const int64_t lane8 = ((ph << p.c.page_shift) + pos) * p.lanes + e8;
    uint8_t* q = value ? a.vq : a.kq;
    if constexpr (kFp4) ((unsigned*)q)[lane8] = out.x;
    else ((u32x2*)q)[lane8] = out;
    if ((e8 & 3) == 0) {
      const int64_t nb = p.c.dim / 32, b = e8 >> 2;
      if (value) a.vs[((ph * nb + b) << p.c.page_shift) + pos] = (uint8_t)code;
      else a.ks[((ph << p.c.page_shift) + pos) * nb + b] = (uint8_t)code;
    }
  }
}

}  // namespace

hipError_t launch_rope_append(const RopeArgs& a, const KvShape& c, bool bf16, bool interleaved, bool fp4,
                              hipStream_t st) {
  RopeParams p;
  p.a = a;
  p.c = c;
  p.lanes = c.dim / 8;
  p.rows = kThreads / p.lanes;
  const unsigned heads = a.q_heads + 2 * c.heads;
  p.tokens = 1;
  while (2 * p.tokens <= p.rows && p.tokens < a.tokens) p.tokens *= 2;
  const unsigned step = p.rows / p.tokens;
  const int64_t runs = (a.tokens + p.tokens - 1) / p.tokens, most = (heads + step - 1) / step;
  // Few runs: as many blocks as fill the chip, down to a head each (256 tokens of 64
  // heads over 8: 8.8 us, with 256 blocks 9.5, with 1024 8.0).  Many: 10 heads a block,
  // enough to share the run's table and few enough that heads of a token are in flight
  // together (16384 tokens: 144 us; all 80 heads 159, 40 157; 2048 tokens 22; 5 heads
  // 29).  Not the best at each size: 4096 tokens take 40 us, with 20 heads 34.
  const int64_t splits = runs >= 128 ? (most + 9) / 10 : std::min(most, 2048 / runs);
  p.heads_each = (unsigned)((most + splits - 1) / splits * step);
  const dim3 grid((unsigned)(runs * ((heads + p.heads_each - 1) / p.heads_each))), block(kThreads);
#define MXQ_ROPE(B, F)                                             \
  interleaved ? k_rope_append<B, F, true><<<grid, block, 0, st>>>(p) \
              : k_rope_append<B, F, false><<<grid, block, 0, st>>>(p)
  if (bf16 && fp4) MXQ_ROPE(true, true);
  else if (bf16) MXQ_ROPE(true, false);
  else if (fp4) MXQ_ROPE(false, true);
  else MXQ_ROPE(false, false);
#undef MXQ_ROPE
  return hipGetLastError();
}

}  // namespace mxq
