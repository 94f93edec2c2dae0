// attention.hip -- attention of one new token per sequence over a paged
// MXFP8 / MXFP4 cache, split over the cache's length and joined (gfx950).
//
//   o = sum_t p_t V_t / (sum_t p_t [+ exp(sink - m)]),  p_t = exp(scale q . K_t - m),
//   t in [max(0, len - window), len), m the running maximum
//
// Mapping.  The query heads that share a cache head are the 16 columns of the
// 16x16x32 bf16 MFMA (more of them: further waves of the block take further
// groups of 16), and a wave walks over tiles of 32 tokens:
//   S^T = K Q^T: K rows as the A operand.  Lane (i = lane & 15, g = lane >> 4)
//     holds token 8 (i / 4) + i % 4 (second product: + 4) and 32 consecutive
//     elements 128 p + 32 g of its row, so its share has one scale and the
//     result puts tokens 8 g .. 8 g + 7 of head i into lane (i, g);
//   O^T += V^T P^T: those eight probabilities ARE the B operand's k slots, so
//     P never crosses lanes.  The A operand is V^T: lane (i, g) loads D / 16
//     consecutive elements of tokens 8 g .. 8 g + 7, and product j takes
//     element j of them (row i <-> d = i D / 16 + j), which turns the
//     transpose of V into byte selects inside the lane.
// Dequantized E4M3 / E2M1 values are exact in bf16.  Scores, maxima, sums and
// O are fp32.  P enters the product as a sum of bf16 terms: two (2^-17 of P)
// for bf16 output, where one term's 2^-9 would add to the output's own
// rounding, and three (2^-25) for fp32 output.
//
// Memory bound: the cache is read once (2 x 1.03 bytes a token, head and
// element in MXFP8, 2 x 0.53 in MXFP4).  A block of 4 waves takes one
// sequence, one cache head and one stretch of the length; partial results
// (m, sum, O) go to the workspace and k_attend_join adds them in order.
#include "mxq_gemm_common.h"
#include "mxq_kv.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kTile = 32;         // tokens a wave takes at a time
constexpr int kWaves = 4;         // waves of a block
constexpr int kMaxPages = 1024;   // page ids a block keeps in LDS
constexpr int kHeadTile = 16;     // query heads of one MFMA column set
constexpr int64_t kMaxLen = 0x7FFFFFC0;  // tokens of a sequence (token indexes are 32 bits)
constexpr float kLog2e = 1.4426950408889634f;

struct AttendParams {
  AttendArgs a;
  KvShape c;
  int splits;       // stretches of the length; the partial results' stride
  unsigned group;   // query heads per cache head
  unsigned tiles16; // head tiles of 16 per cache head
  unsigned tile_groups;  // blocks that share a cache head and stretch
  unsigned block_tiles;  // head tiles a block takes: 1, 2 or 4
  float *part_o, *part_ml;
};

// The stretch of the sequence that split `s` takes, in tiles of 32 tokens.
struct Stretch {
  int first, last;  // tiles [first, last)
  int used;         // splits in use for this sequence
};

__device__ __forceinline__ Stretch stretch(int start, int len, int s, int splits, int min_tiles) {
  const int t0 = start / kTile, t1 = (len + kTile - 1) / kTile;
  const int tiles = t1 - t0;
  int per = (tiles + splits - 1) / splits;
  per = max(per, min_tiles);
  Stretch r;
  r.used = (tiles + per - 1) / per;
  r.first = min(t1, t0 + s * per);
  r.last = min(t1, r.first + per);
  return r;
}

// Visible tokens of a sequence: [start, len).  A length above what the page
// table can name is cut to it.
__device__ __forceinline__ void visible(const AttendArgs& a, const KvShape& c, int64_t b, int& start, int& len) {
  const int64_t most = min(a.table_width << c.page_shift, kMaxLen);
  const int64_t n = min((int64_t)max(a.lens[b], 0), most);
  len = (int)n;
  start = a.window > 0 ? (int)max((int64_t)0, n - a.window) : 0;
}

template <int D, bool kFp4>
struct Tile {
  static constexpr int kRow = kFp4 ? D / 2 : D;       // bytes of a token's row
  static constexpr int kLaneK = kRow / 4;             // bytes of it per lane group
  static constexpr int kLaneV = kRow / 16;            // bytes of it per lane column
  static constexpr int kRuns = D >= 128 ? D / 128 : 1;  // K: pieces of 32 elements a lane holds (D = 64: one of 16)
  unsigned k[2][kLaneK / 4];
  uint8_t ks[2][kRuns];
  unsigned v[8][kLaneV >= 4 ? kLaneV / 4 : 1];
  u32x2 vs;
};

template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, unsigned* o) {
  if constexpr (N == 2) {
    o[0] = *(const uint16_t*)p;
  } else if constexpr (N == 4) {
    o[0] = *(const unsigned*)p;
  } else if constexpr (N == 8) {
    const u32x2 w = *(const u32x2*)p;
    o[0] = w.x, o[1] = w.y;
  } else {
    static_assert(N % 16 == 0);
#pragma unroll
    for (int i = 0; i < N / 16; i++) {
      const u32x4 w = ((const u32x4*)p)[i];
      o[4 * i] = w.x, o[4 * i + 1] = w.y, o[4 * i + 2] = w.z, o[4 * i + 3] = w.w;
    }
  }
}

// K rows of this lane's two tokens.  page: the page of its tokens (0 where
// the tokens are masked), pos: the first token's position in the page.
template <int D, bool kFp4>
__device__ __forceinline__ void load_k(const AttendParams& p, unsigned head, int page, unsigned pos, int g,
                                       Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const int64_t row = (((int64_t)page * p.c.heads + head) << p.c.page_shift) + pos;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const uint8_t* base = p.a.kq + (row + 4 * h) * T::kRow;
    const uint8_t* sb = p.a.ks + (row + 4 * h) * (D / 32);
    if constexpr (D == 64) {
      load_bytes<T::kLaneK>(base + g * T::kLaneK, t.k[h]);
      t.ks[h][0] = sb[g >> 1];
    } else {
      constexpr int kRun = T::kRow / T::kRuns / 4;  // bytes of 32 elements
#pragma unroll
      for (int r = 0; r < T::kRuns; r++) {
        load_bytes<kRun>(base + r * 4 * kRun + g * kRun, t.k[h] + r * kRun / 4);
        t.ks[h][r] = sb[4 * r + g];
      }
    }
  }
}

// V rows of tokens 8 g .. 8 g + 7 (consecutive in one page).
template <int D, bool kFp4>
__device__ __forceinline__ void load_v(const AttendParams& p, unsigned head, int page, unsigned pos, int i,
                                       Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const int64_t ph = (int64_t)page * p.c.heads + head;
  const uint8_t* base = p.a.vq + ((ph << p.c.page_shift) + pos) * T::kRow + i * T::kLaneV;
#pragma unroll
  for (int r = 0; r < 8; r++) load_bytes<T::kLaneV>(base + r * T::kRow, t.v[r]);
  const int blk = i * (D / 16) / 32;
  t.vs = *(const u32x2*)(p.a.vs + ((ph * (D / 32) + blk) << p.c.page_shift) + pos);
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

template <int D, bool kFp4, int kTerms>
__global__ __launch_bounds__(64 * kWaves) void k_attend(AttendParams p, int min_tiles) {
  typedef Tile<D, kFp4> T;
  constexpr int kSteps = D / 32;  // QK products a tile half
  constexpr int J = D / 16;       // PV products a tile; elements of V per lane and token
  constexpr int kPad = D + 4;
  __shared__ union {
    int pages[kMaxPages];
    float o[kWaves][kHeadTile][kPad];
  } lds;
  __shared__ float lds_m[kWaves][kHeadTile], lds_l[kWaves][kHeadTile];

  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // block -> (sequence, split, cache head, head tile group)
  unsigned id = blockIdx.x;
  const unsigned tg = id % p.tile_groups;
  id /= p.tile_groups;
  const unsigned head = id % p.c.heads;
  id /= p.c.heads;
  const int split = (int)(id % (unsigned)p.splits);
  const int64_t b = id / (unsigned)p.splits;

  int start, len;
  visible(p.a, p.c, b, start, len);
  const Stretch st = stretch(start, len, split, p.splits, min_tiles);
  if (st.first >= st.last && !(split == 0)) return;  // split 0 of an empty sequence writes its zeros

  // page ids of the stretch; -1 where the table names no page of the cache
  const unsigned shift = p.c.page_shift;
  const int page0 = (st.first * kTile) >> shift;
  if (st.first < st.last) {
    const int page1 = (min(st.last * kTile, len) - 1) >> shift;
    const int32_t* row = p.a.table + b * p.a.table_stride;
    for (int t = threadIdx.x; t <= page1 - page0; t += 64 * kWaves) {
      const int id0 = row[page0 + t];
      lds.pages[t] = id0 >= 0 && id0 < p.c.pages ? id0 : -1;
    }
  }
  // the wave's head tile, and its place among the waves that share it
  const unsigned per_tile = kWaves / p.block_tiles;  // waves per head tile
  const unsigned tile = tg * p.block_tiles + wave / per_tile;
  const int sub = wave % per_tile;
  const unsigned gh = tile * kHeadTile + i;  // query head of the group in this lane
  const bool live = tile < p.tiles16;
  // Q^T as the B operand: lane (i, g) holds the elements of head i that pair
  // with the K elements of lane group g
  bf16x8 qf[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; s++) {
    const int d = D == 64 ? 16 * g + 8 * s : 128 * (s / 4) + 32 * g + 8 * (s & 3);
    u32x4 w = {0, 0, 0, 0};
    if (live && gh < p.group)
      w = *(const u32x4*)(p.a.q + b * p.a.q_stride + (int64_t)(head * p.group + gh) * D + d);
    qf[s] = __builtin_bit_cast(bf16x8, w);
  }
  __syncthreads();

  float m = -INFINITY, l = 0;
  f32x4 acc[J];
#pragma unroll
  for (int j = 0; j < J; j++) acc[j] = (f32x4){0, 0, 0, 0};
  const float to_log2 = p.a.scale * kLog2e;

  const unsigned pmask = (1u << shift) - 1;
  const int ktok = 8 * (i >> 2) + (i & 3);
  T t;
  int tile_at = st.first + sub;
  int vpage = -1;
  auto page_of = [&](int token) {
    // tokens past the stretch's last page read page 0 and are masked
    const int pg = (token >> shift) - page0;
    return token < len ? lds.pages[pg] : -1;
  };
  if (live && tile_at < st.last) {
    const int k0 = tile_at * kTile + ktok, v0 = tile_at * kTile + 8 * g;
    load_k<D, kFp4>(p, head, max(page_of(k0 & ~7), 0), k0 & pmask, g, t);
    vpage = page_of(v0);
    load_v<D, kFp4>(p, head, max(vpage, 0), v0 & pmask, i, t);
  }
  for (; live && tile_at < st.last; tile_at += per_tile) {
    const int next = tile_at + per_tile;
    const int t0 = tile_at * kTile;
    // S^T
    f32x4 sc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float scale[T::kRuns];
#pragma unroll
      for (int r = 0; r < T::kRuns; r++) scale[r] = e8m0_as_scale(t.ks[h][r]);
#pragma unroll
      for (int s = 0; s < kSteps; s++) {
        const float f = scale[D == 64 ? 0 : s / 4];
        u32x4 a;
#pragma unroll
        for (int e = 0; e < 4; e++) a[e] = decode2<kFp4>(t.k[h], 4 * s + e, f);
        sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), qf[s], sc[h], 0, 0, 0);
      }
    }
    if (next < st.last) {
      const int k0 = next * kTile + ktok;
      load_k<D, kFp4>(p, head, max(page_of(k0 & ~7), 0), k0 & pmask, g, t);
    }
    // softmax over the tile; this lane: head i, tokens t0 + 8 g ..+7
    const int v0 = t0 + 8 * g;
    float x[8];
#pragma unroll
    for (int r = 0; r < 8; r++) x[r] = sc[r >> 2][r & 3] * to_log2;
    const bool whole = t0 >= start && t0 + kTile <= len && __builtin_amdgcn_ballot_w64(vpage < 0) == 0;
    if (!whole) {
      // a masked token's K and V bytes are whatever the page holds: its score
      // is replaced, and its codes and scale are cleared, so nothing of it
      // (NaN codes among it) reaches a product with a non-zero factor
#pragma unroll
      for (int r = 0; r < 8; r++) {
        const bool seen = vpage >= 0 && v0 + r >= start && v0 + r < len;
        x[r] = seen ? x[r] : -INFINITY;
#pragma unroll
        for (int w = 0; w < (int)(sizeof(t.v[r]) / 4); w++) t.v[r][w] = seen ? t.v[r][w] : 0u;
        const unsigned keep = seen ? 0xFFu << (8 * (r & 3)) : 0u;
        const unsigned all = 0xFFu << (8 * (r & 3));
        if (r < 4) t.vs.x &= keep | ~all;
        else t.vs.y &= keep | ~all;
      }
    }
    float top = x[0];
#pragma unroll
    for (int r = 1; r < 8; r++) top = fmaxf(top, x[r]);
    top = fmaxf(m, max_groups(top));
    const float ref = top > -INFINITY ? top : 0.0f;  // nothing seen yet: every p is 0
    if (__builtin_amdgcn_ballot_w64(top > m) != 0) {
      const float alpha = __builtin_amdgcn_exp2f(m - ref);
      l *= alpha;
#pragma unroll
      for (int j = 0; j < J; j++) acc[j] *= alpha;
      m = top;
    }
    u32x4 pt[kTerms];
#pragma unroll
    for (int r = 0; r < 8; r += 2) {
      float p0 = __builtin_amdgcn_exp2f(x[r] - ref), p1 = __builtin_amdgcn_exp2f(x[r + 1] - ref);
      l += p0 + p1;
#pragma unroll
      for (int k = 0; k < kTerms; k++) {
        const unsigned w = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)p0, (__bf16)p1});
        pt[k][r >> 1] = w;
        p0 -= __uint_as_float(w << 16);  // exact: the rest of a rounding
        p1 -= __uint_as_float(w & 0xFFFF0000u);
      }
    }
    // O^T
    float vscale[8];
#pragma unroll
    for (int r = 0; r < 8; r++)
      vscale[r] = e8m0_as_scale((r < 4 ? t.vs.x >> (8 * r) : t.vs.y >> (8 * (r - 4))) & 0xFFu);
#pragma unroll
    for (int j2 = 0; j2 < J / 2; j2++) {
      unsigned d[8];
#pragma unroll
      for (int r = 0; r < 8; r++) d[r] = decode2<kFp4>(t.v[r], j2, vscale[r]);
#pragma unroll
      for (int o = 0; o < 2; o++) {
        u32x4 a;
#pragma unroll
        for (int r = 0; r < 4; r++) a[r] = perm(d[2 * r + 1], d[2 * r], o ? 0x07060302u : 0x05040100u);
        const bf16x8 va = __builtin_bit_cast(bf16x8, a);
#pragma unroll
        for (int k = 0; k < kTerms; k++)
          acc[2 * j2 + o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, __builtin_bit_cast(bf16x8, pt[k]),
                                                                    acc[2 * j2 + o], 0, 0, 0);
      }
    }
    if (next < st.last) {
      const int vn = next * kTile + 8 * g;
      vpage = page_of(vn);
      load_v<D, kFp4>(p, head, max(vpage, 0), vn & pmask, i, t);
    }
  }

  // join the waves of a head tile
  l = sum_groups(l);
  if (g == 0) lds_m[wave][i] = m, lds_l[wave][i] = l;
  __syncthreads();  // also: the page ids are no longer read
  const int w0 = wave - sub;
  float mt = -INFINITY;
  for (unsigned w = 0; w < per_tile; w++) mt = fmaxf(mt, lds_m[w0 + w][i]);
  const float f = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mt) : 0.0f;
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int r = 0; r < 4; r++) lds.o[wave][i][(4 * g + r) * J + j] = acc[j][r] * f;
  __syncthreads();

  // out: lanes of the block over (head tile, head, 4 elements)
  constexpr int kQuads = D / 4;
  const bool direct = st.used <= 1;
  for (int e = threadIdx.x; e < (int)p.block_tiles * kHeadTile * kQuads; e += 64 * kWaves) {
    const int lt = e / (kHeadTile * kQuads), hh = e / kQuads % kHeadTile, d4 = e % kQuads;
    const unsigned gq = (tg * p.block_tiles + lt) * kHeadTile + hh;
    if (gq >= p.group) continue;
    const int wb = lt * per_tile;
    float mx = -INFINITY;
    for (unsigned w = 0; w < per_tile; w++) mx = fmaxf(mx, lds_m[wb + w][hh]);
    float sum = 0;
    f32x4 o = {0, 0, 0, 0};
    for (unsigned w = 0; w < per_tile; w++) {
      const float mw = lds_m[wb + w][hh];
      sum += mw > -INFINITY ? lds_l[wb + w][hh] * __builtin_amdgcn_exp2f(mw - mx) : 0.0f;
      o += *(const f32x4*)&lds.o[wb + w][hh][4 * d4];
    }
    const int64_t hq = (int64_t)head * p.group + gq;
    const int64_t bh = b * p.a.q_heads + hq;
    if (direct) {
      if (p.a.sinks && mx > -INFINITY) {
        const float sk = p.a.sinks[hq] * kLog2e, top = fmaxf(mx, sk);
        const float fx = __builtin_amdgcn_exp2f(mx - top);
        sum = sum * fx + __builtin_amdgcn_exp2f(sk - top);
        o *= fx;
      }
      o = sum > 0 ? o / sum : (f32x4){0, 0, 0, 0};
      const int64_t at = bh * D + 4 * d4;
      if (p.a.bf16_out) {
        const unsigned x0 = f32_to_bf16_rne(o[0]) | ((unsigned)f32_to_bf16_rne(o[1]) << 16);
        const unsigned x1 = f32_to_bf16_rne(o[2]) | ((unsigned)f32_to_bf16_rne(o[3]) << 16);
        *(u32x2*)((uint16_t*)p.a.out + at) = (u32x2){x0, x1};
      } else {
        *(f32x4*)((float*)p.a.out + at) = o;
      }
    } else {
      const int64_t slot = bh * p.splits + split;
      *(f32x4*)(p.part_o + slot * D + 4 * d4) = o;
      if (d4 == 0) {
        p.part_ml[2 * slot] = mx;
        p.part_ml[2 * slot + 1] = sum;
      }
    }
  }
}

// Adds the partial results of one sequence and query head, in the order of
// the splits inside each of the block's 256 / (D / 4) rows, then row by row.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p, int min_tiles) {
  constexpr int kQuads = D / 4, kRows = 256 / kQuads;
  __shared__ f32x4 lo[kRows][kQuads];
  __shared__ float ll[kRows];
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / p.a.q_heads;
  const unsigned hq = (unsigned)(bh % p.a.q_heads);
  int start, len;
  visible(p.a, p.c, b, start, len);
  const Stretch st = stretch(start, len, 0, p.splits, min_tiles);
  if (st.used <= 1) return;  // written by k_attend
  const int d4 = threadIdx.x % kQuads, row = threadIdx.x / kQuads;
  const float* ml = p.part_ml + 2 * bh * p.splits;
  const f32x4* po = (const f32x4*)(p.part_o + bh * p.splits * D);
  float top = p.a.sinks ? p.a.sinks[hq] * kLog2e : -INFINITY;
  bool any = false;
  for (int s = 0; s < st.used; s++) {
    any |= ml[2 * s] > -INFINITY;
    top = fmaxf(top, ml[2 * s]);
  }
  f32x4 o = {0, 0, 0, 0};
  float sum = 0;
  for (int s = row; s < st.used; s += kRows) {
    const float mw = ml[2 * s];
    const float f = mw > -INFINITY ? __builtin_amdgcn_exp2f(mw - top) : 0.0f;
    sum += f * ml[2 * s + 1];
    o += po[(int64_t)s * kQuads + d4] * f;
  }
  lo[row][d4] = o;
  if (d4 == 0) ll[row] = sum;
  __syncthreads();
  if (row != 0) return;
  for (int r = 1; r < kRows; r++) {
    o += lo[r][d4];
    sum += ll[r];
  }
  if (p.a.sinks && any) sum += __builtin_amdgcn_exp2f(p.a.sinks[hq] * kLog2e - top);
  o = any && sum > 0 ? o / sum : (f32x4){0, 0, 0, 0};
  const int64_t at = bh * D + 4 * d4;
  if (p.a.bf16_out) {
    const unsigned x0 = f32_to_bf16_rne(o[0]) | ((unsigned)f32_to_bf16_rne(o[1]) << 16);
    const unsigned x1 = f32_to_bf16_rne(o[2]) | ((unsigned)f32_to_bf16_rne(o[3]) << 16);
    *(u32x2*)((uint16_t*)p.a.out + at) = (u32x2){x0, x1};
  } else {
    *(f32x4*)((float*)p.a.out + at) = o;
  }
}

constexpr int kMinTiles = kWaves;      // a stretch gives every wave a tile
constexpr int kTargetBlocks = 1024;    // four blocks a CU

}  // namespace

// Head tiles of 16 per cache head, and the blocks that share its cache: a
// block's four waves take up to four head tiles.
static int64_t head_tiles(unsigned q_heads, const KvShape& c) { return (q_heads / c.heads + kHeadTile - 1) / kHeadTile; }
static int64_t tile_groups(unsigned q_heads, const KvShape& c) { return (head_tiles(q_heads, c) + kWaves - 1) / kWaves; }

static int attend_splits(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  int64_t most = std::min<int64_t>(table_width << c.page_shift, kMaxLen);
  if (window > 0 && window < most) most = std::min(most, window + kTile);
  const int64_t tiles = std::max<int64_t>(1, (most + kTile - 1) / kTile);
  const int64_t units = batch * c.heads * tile_groups(q_heads, c);
  int64_t s = (kTargetBlocks + units - 1) / units;
  s = std::min(s, (tiles + kMinTiles - 1) / kMinTiles);
  // the page ids of a stretch fit the block's LDS
  const int64_t tiles_most = std::max<int64_t>(1, ((int64_t)(kMaxPages - 2) << c.page_shift) / kTile);
  s = std::max(s, (tiles + tiles_most - 1) / tiles_most);
  return (int)std::max<int64_t>(1, s);
}

int64_t attend_blocks(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  return batch * attend_splits(batch, q_heads, c, table_width, window) * c.heads * tile_groups(q_heads, c);
}

int64_t attend_workspace(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  const int64_t s = attend_splits(batch, q_heads, c, table_width, window);
  return s == 1 ? 0 : batch * q_heads * s * (int64_t)(c.dim + 2) * 4;
}

hipError_t launch_attend(const AttendArgs& a, const KvShape& c, bool fp4, void* workspace, hipStream_t st) {
  AttendParams p;
  p.a = a;
  p.c = c;
  p.splits = attend_splits(a.batch, a.q_heads, c, a.table_width, a.window);
  p.group = a.q_heads / c.heads;
  p.tiles16 = (unsigned)head_tiles(a.q_heads, c);
  p.block_tiles = p.tiles16 >= 3 ? 4 : p.tiles16;
  p.tile_groups = (unsigned)tile_groups(a.q_heads, c);
  p.part_o = (float*)workspace;
  p.part_ml = p.part_o + a.batch * a.q_heads * p.splits * (int64_t)c.dim;
  const dim3 grid((unsigned)attend_blocks(a.batch, a.q_heads, c, a.table_width, a.window)), block(64 * kWaves);
#define MXQ_ATTEND_T(D, T) \
  fp4 ? k_attend<D, true, T><<<grid, block, 0, st>>>(p, kMinTiles) : k_attend<D, false, T><<<grid, block, 0, st>>>(p, kMinTiles)
#define MXQ_ATTEND(D)                                                                                            \
  do {                                                                                                           \
    if (a.bf16_out) MXQ_ATTEND_T(D, 2);                                                                          \
    else MXQ_ATTEND_T(D, 3);                                                                                     \
    if (p.splits > 1) k_attend_join<D><<<dim3((unsigned)(a.batch * a.q_heads)), dim3(256), 0, st>>>(p, kMinTiles); \
  } while (0)
  if (c.dim == 64) MXQ_ATTEND(64);
  else if (c.dim == 128) MXQ_ATTEND(128);
  else MXQ_ATTEND(256);
#undef MXQ_ATTEND
#undef MXQ_ATTEND_T
  return hipGetLastError();
}

}  // namespace mxq
