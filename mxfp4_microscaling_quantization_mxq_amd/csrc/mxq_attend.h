// mxq_attend.h -- device code that the attention kernels over the paged cache
// share: a tile of 32 tokens as loaded, its loads and decoding, and the end of a
// row (gfx950).
#pragma once
#include "mxq_gemm_common.h"
#include "mxq_kv.h"
#include "mxq_launch.h"

namespace mxq {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;  // tokens a wave takes at a time
constexpr int64_t kMaxLen = 0x7FFF0000;  // tokens of a sequence (token indexes, also a few tiles past it, are 32 bits)
constexpr float kLog2e = 1.4426950408889634f;

// The compiler keeps what it cannot prove to be the same in every lane in
// vector registers; loop bounds and addresses are scalar only with this.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int D, bool kFp4>
struct Tile {
  static constexpr int kRow = kFp4 ? D / 2 : D;         // bytes of a token's row
  static constexpr int kRuns = D >= 128 ? D / 128 : 1;  // K: pieces of 32 elements a lane holds (D = 64: one of 16)
  static constexpr int kRun = kRow / 4 / kRuns;         // bytes of one
  static constexpr int kLaneV = kRow / 16;              // V: bytes of a token a lane holds
  unsigned k[2][kRuns * kRun / 4], v[8][kLaneV >= 4 ? kLaneV / 4 : 1];
  uint8_t ks[2][kRuns];
  unsigned vs[2];
};

// Loads of the cache's codes: each byte is read by one wave (or by the waves
// of one block), so they carry the streaming hint (2).
template <int N>
__device__ __forceinline__ void load_bytes(__amdgpu_buffer_rsrc_t r, int off, unsigned* o) {
  if constexpr (N == 2) {
    o[0] = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 2);
  } else if constexpr (N == 4) {
    o[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 2);
  } else if constexpr (N == 8) {
    const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 2);
    o[0] = w.x, o[1] = w.y;
  } else {
    static_assert(N % 16 == 0);
#pragma unroll
    for (int i = 0; i < N / 16; i++) {
      const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 2);
      o[4 * i] = w.x, o[4 * i + 1] = w.y, o[4 * i + 2] = w.z, o[4 * i + 3] = w.w;
    }
  }
}

// Where 16 consecutive tokens of one cache head lie: row `row` of the cache,
// (page * heads + head) * P + position, or nowhere (on = false).
struct Half {
  int64_t row;
  bool on;
};
template <int D, bool kFp4, class Params>
__device__ __forceinline__ void load_k(const Params& p, Half f, int h, int i, int g, Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const __amdgpu_buffer_rsrc_t rq = panel_rsrc(p.a.kq + f.row * T::kRow, f.on ? 16 * T::kRow : 0);
  const __amdgpu_buffer_rsrc_t rs = panel_rsrc(p.a.ks + f.row * (D / 32), f.on ? 16 * (D / 32) : 0);
#pragma unroll
  for (int r = 0; r < T::kRuns; r++) {
    load_bytes<T::kRun>(rq, i * T::kRow + g * T::kRun + r * 4 * T::kRun, t.k[h] + r * T::kRun / 4);
    t.ks[h][r] = __builtin_amdgcn_raw_buffer_load_b8(rs, i * (D / 32) + (D == 64 ? g >> 1 : g + 4 * r), 0, 0);
  }
}
template <int D, bool kFp4, class Params>
__device__ __forceinline__ void load_v(const Params& p, Half f, unsigned pos, int h, int i, int g,
                                       Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const unsigned shift = p.c.page_shift;
  const __amdgpu_buffer_rsrc_t rq = panel_rsrc(p.a.vq + f.row * T::kRow, f.on ? 16 * T::kRow : 0);
  const __amdgpu_buffer_rsrc_t rs =
      panel_rsrc(p.a.vs + (f.row - pos) * (D / 32) + pos, f.on ? ((D / 32 - 1) << shift) + 16 : 0);
#pragma unroll
  for (int r = 0; r < 4; r++) load_bytes<T::kLaneV>(rq, 4 * g * T::kRow + i * T::kLaneV + r * T::kRow, t.v[4 * h + r]);
  const int blk = i * (D / 16) / 32;
  t.vs[h] = __builtin_amdgcn_raw_buffer_load_b32(rs, (blk << shift) + 4 * g, 0, 0);
}

__device__ __forceinline__ unsigned perm(unsigned hi, unsigned lo, unsigned sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

// Two elements (2 e, 2 e + 1 of the dword-packed codes w) times scale, bf16.
template <bool kFp4>
__device__ __forceinline__ unsigned decode2(const unsigned* w, int e, float scale) {
  bf16x2 r;
  if constexpr (kFp4) {
    switch (e & 3) {
      case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[e >> 2], scale, 0); break;
      case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[e >> 2], scale, 1); break;
      case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[e >> 2], scale, 2); break;
      default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[e >> 2], scale, 3); break;
    }
  } else {
    if (e & 1) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e >> 1], scale, true);
    else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[e >> 1], scale, false);
  }
  return __builtin_bit_cast(unsigned, r);
}

// Largest value over the four lane groups, in every lane.
__device__ __forceinline__ float max_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Stores four elements of the output.
template <class Args>
__device__ __forceinline__ void store_out(const Args& a, int64_t at, f32x4 o) {
  if (a.bf16_out) {
    const unsigned x0 = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)o[0], (__bf16)o[1]});
    const unsigned x1 = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)o[2], (__bf16)o[3]});
    *(u32x2*)((uint16_t*)a.out + at) = (u32x2){x0, x1};
  } else {
    *(f32x4*)((float*)a.out + at) = o;
  }
}

// Partial results of one unit: m is in units of the scores' log2.
// o = sum_t 2^(x_t - m) V_t and sum likewise -> the output, with the head's sink.
template <class Args>
__device__ __forceinline__ f32x4 finish(const Args& a, int64_t hq, float m, float sum, f32x4 o) {
  // Nothing visible.  (Scores that are all NaN leave m there too, and a NaN sum.)
  if (!(m > -INFINITY) && sum == 0) return (f32x4){0, 0, 0, 0};
  if (a.sinks) {
    const float sk = a.sinks[hq] * kLog2e, top = fmaxf(m, sk), f = __builtin_amdgcn_exp2f(m - top);
    sum = sum * f + __builtin_amdgcn_exp2f(sk - top);
    o *= f;
  }
  return o / sum;
}

}  // namespace mxq
