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
// element in MXFP8, 2 x 0.53 in MXFP4).
//
// Split.  A unit is one sequence and one cache head (and up to 64 of its query
// heads); its work is its visible tiles.  The tiles of all units, in order,
// are cut into equal ranges, one a block of 4 waves, so a batch of uneven
// lengths keeps every CU busy to the end.  A range that ends inside a unit
// leaves partial results (m, sum, O) in the workspace, and k_attend_join adds
// a unit's parts in order.  Where no unit is long and there are many, a block
// takes one unit and nothing is joined.
#include "mxq_gemm_common.h"
#include "mxq_kv.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

constexpr int kTile = 32;       // tokens a wave takes at a time
constexpr int kWaves = 4;       // waves of a block
constexpr int kThreads = 64 * kWaves;
constexpr int kHeadTile = 16;   // query heads of one MFMA column set
constexpr int64_t kMaxLen = 0x7FFFFFC0;  // tokens of a sequence (token indexes are 32 bits)
constexpr float kLog2e = 1.4426950408889634f;

struct AttendParams {
  AttendArgs a;
  KvShape c;
  unsigned group;        // query heads per cache head
  unsigned tiles16;      // head tiles of 16 per cache head
  unsigned tile_groups;  // units per sequence and cache head
  unsigned block_tiles;  // head tiles of a unit: 1, 2 or 4
  bool ranges;           // blocks take ranges of the flattened list, or one unit each
  unsigned* first;       // [batch + 1] first flattened tile of each sequence, then their sum
  float *part_o, *part_ml;  // [2 blocks][16 block_tiles][D], [2 blocks][16 block_tiles][2]
};

// Visible tokens of a sequence: [start, len), in tiles [t0, t1).  A length
// above what the page table can name is cut to it.
struct Span {
  int start, len, t0, t1;
};
__device__ __forceinline__ Span span_tiles(int start, int len) {
  return {start, len, (int)((unsigned)start / kTile), (int)(((unsigned)len + kTile - 1) / kTile)};
}
__device__ __forceinline__ Span span_of(const AttendParams& p, int64_t b) {
  const int64_t most = min(p.a.table_width << p.c.page_shift, kMaxLen);
  const int64_t n = min((int64_t)max(p.a.lens[b], 0), most);
  return span_tiles(p.a.window > 0 ? (int)max((int64_t)0, n - p.a.window) : 0, (int)n);
}

// Tiles of a range for a sum of all tiles: an equal share of each of 2^9
// blocks (two a CU), and enough to give every wave one.
constexpr int kRangeShift = 9;
__device__ __forceinline__ unsigned range_tiles(unsigned sum) {
  return max((sum >> kRangeShift) + ((sum & ((1u << kRangeShift) - 1)) != 0), (unsigned)kWaves);
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

// Each byte of the cache is read by one wave (or by the waves of one block),
// so the loads carry the streaming hint.
template <int N>
__device__ __forceinline__ void load_bytes(const uint8_t* p, unsigned* o) {
  if constexpr (N == 2) {
    o[0] = __builtin_nontemporal_load((const uint16_t*)p);
  } else if constexpr (N == 4) {
    o[0] = __builtin_nontemporal_load((const unsigned*)p);
  } else if constexpr (N == 8) {
    const u32x2 w = __builtin_nontemporal_load((const u32x2*)p);
    o[0] = w.x, o[1] = w.y;
  } else {
    static_assert(N % 16 == 0);
#pragma unroll
    for (int i = 0; i < N / 16; i++) {
      const u32x4 w = __builtin_nontemporal_load(&((const u32x4*)p)[i]);
      o[4 * i] = w.x, o[4 * i + 1] = w.y, o[4 * i + 2] = w.z, o[4 * i + 3] = w.w;
    }
  }
}

// K rows of this lane's two tokens: rows `row` and `row` + 4 of a page that
// starts at kq (codes) and ks (scales).
template <int D, bool kFp4>
__device__ __forceinline__ void load_k(const uint8_t* kq, const uint8_t* ks, unsigned row, int g, Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const uint8_t* base = kq + (row + 4 * h) * T::kRow;
    const uint8_t* sb = ks + (row + 4 * h) * (D / 32);
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

// V rows `row` .. `row` + 7 of a page that starts at vq (codes) and vs (scales).
template <int D, bool kFp4>
__device__ __forceinline__ void load_v(const uint8_t* vq, const uint8_t* vs, unsigned row, unsigned shift, int i,
                                       Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const uint8_t* base = vq + row * T::kRow + i * T::kLaneV;
#pragma unroll
  for (int r = 0; r < 8; r++) load_bytes<T::kLaneV>(base + r * T::kRow, t.v[r]);
  const unsigned blk = i * (D / 16) / 32;
  t.vs = *(const u32x2*)(vs + (blk << shift) + row);
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
__device__ __forceinline__ void store_out(const AttendArgs& a, int64_t at, f32x4 o) {
  if (a.bf16_out) {
    const unsigned x0 = f32_to_bf16_rne(o[0]) | ((unsigned)f32_to_bf16_rne(o[1]) << 16);
    const unsigned x1 = f32_to_bf16_rne(o[2]) | ((unsigned)f32_to_bf16_rne(o[3]) << 16);
    *(u32x2*)((uint16_t*)a.out + at) = (u32x2){x0, x1};
  } else {
    *(f32x4*)((float*)a.out + at) = o;
  }
}

// Partial results of one unit: m is in units of the scores' log2.
// o = sum_t 2^(x_t - m) V_t and sum likewise -> the output, with the head's sink.
__device__ __forceinline__ f32x4 finish(const AttendArgs& a, int64_t hq, float m, float sum, f32x4 o) {
  if (!(m > -INFINITY)) return (f32x4){0, 0, 0, 0};  // nothing visible
  if (a.sinks) {
    const float sk = a.sinks[hq] * kLog2e, top = fmaxf(m, sk), f = __builtin_amdgcn_exp2f(m - top);
    sum = sum * f + __builtin_amdgcn_exp2f(sk - top);
    o *= f;
  }
  return o / sum;
}

// Occupancy 2 (blocks a CU): eight waves keep the memory busy, and with at
// most 256 registers a wave the accumulators stay out of the AGPR file, whose
// moves would cost 64 instructions a tile.
template <int D, bool kFp4, int kTerms>
__global__ __launch_bounds__(kThreads, 2) void k_attend(AttendParams p) {
  typedef Tile<D, kFp4> T;
  constexpr int kSteps = D / 32;  // QK products of half a tile
  constexpr int J = D / 16;       // PV products of a tile; elements of V per lane and token
  constexpr int kPad = D + 4;
  constexpr int kBuf = D == 256 ? 1 : 2;  // tiles a wave has on their way
  __shared__ float lds_o[kWaves][kHeadTile][kPad];
  __shared__ float lds_m[kWaves][kHeadTile], lds_l[kWaves][kHeadTile];
  __shared__ unsigned lds_sum[kWaves];
  __shared__ int lds_at[5];

  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // This block's tiles: [x, end) of the flattened list, starting in unit
  // (b, head, tile group tg), whose first tile is u_first.
  unsigned x, end, u_first, head, tg;
  int64_t b;
  Span s;
  if (!p.ranges) {
    unsigned id = blockIdx.x;
    tg = id % p.tile_groups;
    id /= p.tile_groups;
    head = id % p.c.heads;
    b = id / p.c.heads;
    s = span_of(p, b);
    x = u_first = 0;
    end = s.t1 - s.t0;
    if (end == 0) {  // an empty sequence: its zeros
      const unsigned h0 = tg * p.block_tiles * kHeadTile, n = min(p.group - h0, p.block_tiles * kHeadTile);
      const int64_t at = (b * p.a.q_heads + head * p.group + h0) * D;
      for (unsigned e = threadIdx.x; e < n * (D / 4); e += kThreads) store_out(p.a, at + 4 * e, (f32x4){0, 0, 0, 0});
      return;
    }
  } else {
    // each thread sums the tiles of a run of sequences; scan over the block
    const unsigned units = p.c.heads * p.tile_groups;  // of a sequence
    const unsigned batch = (unsigned)p.a.batch, each = (batch + kThreads - 1) / kThreads;
    const unsigned b0 = min(threadIdx.x * each, batch), b1 = min(b0 + each, batch);
    unsigned own = 0;
    for (unsigned k = b0; k < b1; k++) {
      s = span_of(p, k);
      own += (s.t1 - s.t0) * units;
    }
    unsigned incl = own;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const unsigned o = __shfl_up(incl, m, 64);
      if (lane >= m) incl += o;
    }
    if (lane == 63) lds_sum[wave] = incl;
    __syncthreads();
    unsigned sum = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      if (w < wave) before += lds_sum[w];
      sum += lds_sum[w];
    }
    const unsigned per = range_tiles(sum);
    x = blockIdx.x * per;
    end = min(x + per, sum);
    unsigned at = before + incl - own;  // first tile of this thread's sequences
    if (blockIdx.x == 0 || (x >= at && x < at + own)) {
      for (unsigned k = b0; k < b1; k++) {
        if (blockIdx.x == 0) p.first[k] = at;
        s = span_of(p, k);
        const unsigned n = s.t1 - s.t0;
        if (x >= at && x < at + n * units) {
          const unsigned u = (x - at) / n;
          lds_at[0] = (int)k, lds_at[1] = (int)u, lds_at[2] = (int)(at + u * n), lds_at[3] = s.start, lds_at[4] = s.len;
        }
        at += n * units;
      }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.first[batch] = sum;
    if (x >= end) return;
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(lds_at[0]);
    const unsigned u = __builtin_amdgcn_readfirstlane(lds_at[1]);
    u_first = __builtin_amdgcn_readfirstlane(lds_at[2]);
    s = span_tiles(__builtin_amdgcn_readfirstlane(lds_at[3]), __builtin_amdgcn_readfirstlane(lds_at[4]));
    head = u / p.tile_groups;
    tg = u % p.tile_groups;
  }

  const unsigned per_tile = kWaves / p.block_tiles;  // waves per head tile
  const int sub = wave % per_tile;                   // this wave among them
  const unsigned shift = p.c.page_shift, pmask = (1u << shift) - 1;
  const int ktok = 8 * (i >> 2) + (i & 3);
  // scores are scaled by |scale| (its sign is in q), never by less than what
  // keeps a masked score at -inf
  const float to_log2 = fmaxf(fabsf(p.a.scale) * kLog2e, 0x1p-100f);
  const unsigned q_sign = p.a.scale < 0 ? 0x80008000u : 0u;

  while (true) {
    // tiles [first, last) of the unit
    const int first = s.t0 + (int)(x - u_first), last = min(s.t1, s.t0 + (int)(end - u_first));
    const unsigned h0 = tg * p.block_tiles * kHeadTile;  // first query head of the unit

    // Q^T as the B operand: lane (i, g) holds the elements of head i that pair
    // with the K elements of lane group g
    const unsigned gh = h0 + wave / per_tile * kHeadTile + i;
    const bool live = h0 + wave / per_tile * kHeadTile < p.group;
    bf16x8 qf[kSteps];
#pragma unroll
    for (int st = 0; st < kSteps; st++) {
      const int d = D == 64 ? 16 * g + 8 * st : 128 * (st / 4) + 32 * g + 8 * (st & 3);
      u32x4 w = {0, 0, 0, 0};
      if (gh < p.group) w = *(const u32x4*)(p.a.q + b * p.a.q_stride + (int64_t)(head * p.group + gh) * D + d);
      qf[st] = __builtin_bit_cast(bf16x8, w ^ q_sign);
    }

    float m = -INFINITY, l = 0;  // of the unscaled scores, and of this lane's tokens
    f32x4 acc[J];
#pragma unroll
    for (int j = 0; j < J; j++) acc[j] = (f32x4){0, 0, 0, 0};

    // This wave's tiles are first + sub + per_tile j.  Lane k keeps the page ids
    // of tile 64 q + k (two where a tile spans two pages of 16), -1 where the
    // table names no page of the cache; the ids of the next 64 tiles are
    // loaded while these are in use.
    const int32_t* row = p.a.table + b * p.a.table_stride;
    const bool pair = shift == 4;
    auto load_ids = [&](int j, int& ia, int& ib) {
      const int64_t tile = first + sub + (int64_t)per_tile * j;
      ia = ib = -1;
      if (live && tile < last) {
        const int tok = (int)tile * kTile;
        ia = row[tok >> shift];
        if (pair && tok + 16 < s.len) ib = row[(tok + 16) >> shift];
        ia = ia >= 0 && ia < p.c.pages ? ia : -1;
        ib = ib >= 0 && ib < p.c.pages ? ib : -1;
      }
    };
    int ids_a, ids_b, next_a, next_b;
    load_ids(lane, ids_a, ids_b);
    load_ids(64 + lane, next_a, next_b);
    int fetched = 0;  // tiles whose K is on its way

    T t[kBuf];
    int page_a[kBuf], page_b[kBuf];  // of the tile in each buffer
    // rows of a page; a tile (or half of one) without a page reads page 0 and is masked
    auto row_of = [&](int page) { return ((int64_t)max(page, 0) * p.c.heads + head) << shift; };
    auto fetch_k = [&](T& tb, int& pa, int& pb) {
      if ((fetched & 63) == 0 && fetched > 0) {
        ids_a = next_a, ids_b = next_b;
        load_ids(fetched + 64 + lane, next_a, next_b);
      }
      pa = __builtin_amdgcn_readlane(ids_a, fetched & 63);
      const int tok = (first + sub + (int)per_tile * fetched) * kTile;
      if (!pair) {  // one page a tile: scalar addresses
        const int64_t r = row_of(pa) + (tok & pmask);
        load_k<D, kFp4>(p.a.kq + r * T::kRow, p.a.ks + r * (D / 32), ktok, g, tb);
      } else {
        pb = __builtin_amdgcn_readlane(ids_b, fetched & 63);
        const int64_t ra = row_of(pa), rb = row_of(pb), r = ktok < 16 ? ra : rb;
        load_k<D, kFp4>(p.a.kq + r * T::kRow, p.a.ks + r * (D / 32), ktok & 15, g, tb);
      }
      fetched++;
    };
    auto fetch_v = [&](int tile, T& tb, int pa, int pb) {
      if (!pair) {
        const int64_t r = row_of(pa);
        const unsigned pos = (tile * kTile) & pmask;
        load_v<D, kFp4>(p.a.vq + (r + pos) * T::kRow, p.a.vs + r * (D / 32) + pos, 8 * g, shift, i, tb);
      } else {
        const int64_t ra = row_of(pa), rb = row_of(pb), r = g < 2 ? ra : rb;
        load_v<D, kFp4>(p.a.vq + r * T::kRow, p.a.vs + r * (D / 32), 8 * (g & 1), shift, i, tb);
      }
    };
#pragma unroll
    for (int bf = 0; bf < kBuf; bf++) {
      const int at = first + sub + (int)per_tile * bf;
      page_a[bf] = page_b[bf] = -1;
      if (live && at < last) {
        fetch_k(t[bf], page_a[bf], page_b[bf]);
        fetch_v(at, t[bf], page_a[bf], page_b[bf]);
      }
    }
    for (int at0 = first + sub; live && at0 < last; at0 += kBuf * per_tile) {
#pragma unroll
      for (int bf = 0; bf < kBuf; bf++) {
        const int at = at0 + bf * (int)per_tile;
        if (at >= last) break;
        T& tb = t[bf];
        const int next = at + kBuf * (int)per_tile;
        const int t0 = at * kTile;
        const int vpage = pair && g >= 2 ? page_b[bf] : page_a[bf];  // of tokens 8 g .. 8 g + 7
        // S^T
        f32x4 sc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float scale[T::kRuns];
#pragma unroll
          for (int r = 0; r < T::kRuns; r++) scale[r] = e8m0_as_scale(tb.ks[h][r]);
#pragma unroll
          for (int st = 0; st < kSteps; st++) {
            u32x4 a;
#pragma unroll
            for (int e = 0; e < 4; e++) a[e] = decode2<kFp4>(tb.k[h], 4 * st + e, scale[D == 64 ? 0 : st / 4]);
            sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), qf[st], sc[h], 0, 0, 0);
          }
        }
        if (next < last) fetch_k(tb, page_a[bf], page_b[bf]);
        // softmax over the tile; this lane: head i, tokens t0 + 8 g ..+7
        const int v0 = t0 + 8 * g;
        float y[8];
#pragma unroll
        for (int r = 0; r < 8; r++) y[r] = sc[r >> 2][r & 3];
        const bool whole = t0 >= s.start && t0 + kTile <= s.len && __builtin_amdgcn_ballot_w64(vpage < 0) == 0;
        if (!whole) {
          // a masked token's K and V bytes are whatever the page holds: its
          // score is replaced, and its codes and scale are cleared, so nothing
          // of it (NaN codes among it) reaches a product with a non-zero factor
#pragma unroll
          for (int r = 0; r < 8; r++) {
            const bool seen = vpage >= 0 && v0 + r >= s.start && v0 + r < s.len;
            y[r] = seen ? y[r] : -INFINITY;
#pragma unroll
            for (int w = 0; w < (int)(sizeof(tb.v[r]) / 4); w++) tb.v[r][w] = seen ? tb.v[r][w] : 0u;
            const unsigned byte = 0xFFu << (8 * (r & 3));
            if (r < 4) tb.vs.x = seen ? tb.vs.x : tb.vs.x & ~byte;
            else tb.vs.y = seen ? tb.vs.y : tb.vs.y & ~byte;
          }
        }
        float top = y[0];
#pragma unroll
        for (int r = 1; r < 8; r++) top = fmaxf(top, y[r]);
        top = fmaxf(m, max_groups(top));
        const float ref = top > -INFINITY ? top * to_log2 : 0.0f;  // nothing seen yet: every p is 0
        if (__builtin_amdgcn_ballot_w64(top > m) != 0) {
          const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf(m, to_log2, -ref));
          l *= alpha;
#pragma unroll
          for (int j = 0; j < J; j++) acc[j] *= alpha;
          m = top;
        }
        // P in bf16 terms: each takes the upper half of what the ones before
        // it left (truncated; the last one rounded)
        u32x4 pt[kTerms];
#pragma unroll
        for (int r = 0; r < 8; r += 2) {
          float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(y[r], to_log2, -ref));
          float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(y[r + 1], to_log2, -ref));
          l += p0 + p1;
#pragma unroll
          for (int k = 0; k < kTerms; k++) {
            if (k + 1 == kTerms) {
              pt[k][r >> 1] = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)p0, (__bf16)p1});
            } else {
              const unsigned w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
              pt[k][r >> 1] = perm(w1, w0, 0x07060302u);
              p0 -= __uint_as_float(w0 & 0xFFFF0000u);  // exact
              p1 -= __uint_as_float(w1 & 0xFFFF0000u);
            }
          }
        }
        // O^T
        float vscale[8];
#pragma unroll
        for (int r = 0; r < 8; r++)
          vscale[r] = e8m0_as_scale((r < 4 ? tb.vs.x >> (8 * r) : tb.vs.y >> (8 * (r - 4))) & 0xFFu);
#pragma unroll
        for (int j2 = 0; j2 < J / 2; j2++) {
          unsigned d[8];
#pragma unroll
          for (int r = 0; r < 8; r++) d[r] = decode2<kFp4>(tb.v[r], j2, vscale[r]);
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
        if (next < last) fetch_v(next, tb, page_a[bf], page_b[bf]);
      }
    }

    // join the waves of a head tile (maxima in log2 units from here on)
    l = sum_groups(l);
    m *= to_log2;
    if (g == 0) lds_m[wave][i] = m, lds_l[wave][i] = l;
    __syncthreads();
    const int w0 = wave - sub;
    float mt = -INFINITY;
    for (unsigned w = 0; w < per_tile; w++) mt = fmaxf(mt, lds_m[w0 + w][i]);
    const float f = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mt) : 0.0f;
#pragma unroll
    for (int j = 0; j < J; j++)
#pragma unroll
      for (int r = 0; r < 4; r++) lds_o[wave][i][(4 * g + r) * J + j] = acc[j][r] * f;
    __syncthreads();

    // out: threads over (head tile, head, 4 elements)
    constexpr int kQuads = D / 4;
    const bool opens = first == s.t0, closes = last == s.t1;  // of the unit
    for (unsigned e = threadIdx.x; e < p.block_tiles * kHeadTile * kQuads; e += kThreads) {
      const unsigned hh = e / kQuads, d4 = e % kQuads;  // head of the unit
      if (h0 + hh >= p.group) continue;
      const unsigned wb = hh / kHeadTile * per_tile;
      float mx = -INFINITY;
      for (unsigned w = 0; w < per_tile; w++) mx = fmaxf(mx, lds_m[wb + w][hh % kHeadTile]);
      float sum = 0;
      f32x4 o = {0, 0, 0, 0};
      for (unsigned w = 0; w < per_tile; w++) {
        const float mw = lds_m[wb + w][hh % kHeadTile];
        sum += mw > -INFINITY ? lds_l[wb + w][hh % kHeadTile] * __builtin_amdgcn_exp2f(mw - mx) : 0.0f;
        o += *(const f32x4*)&lds_o[wb + w][hh % kHeadTile][4 * d4];
      }
      if (opens && closes) {
        const int64_t hq = (int64_t)head * p.group + h0 + hh;
        store_out(p.a, (b * p.a.q_heads + hq) * D + 4 * d4, finish(p.a, hq, mx, sum, o));
      } else {
        // a block has at most one part of a unit that a block before it
        // opened (slot 0) and one of a unit that it opens itself (slot 1)
        const int64_t slot = (2 * (int64_t)blockIdx.x + (opens ? 1 : 0)) * (p.block_tiles * kHeadTile) + hh;
        *(f32x4*)(p.part_o + slot * D + 4 * d4) = o;
        if (d4 == 0) {
          p.part_ml[2 * slot] = mx;
          p.part_ml[2 * slot + 1] = sum;
        }
      }
    }
    // the next unit: the next tile group, cache head or sequence with tiles
    x = u_first + (last - s.t0);
    if (x >= end) break;
    u_first = x;
    if (++tg == p.tile_groups) {
      tg = 0;
      if (++head == p.c.heads) {
        head = 0;
        do s = span_of(p, ++b);
        while (s.t0 == s.t1);
      }
    }
    __syncthreads();  // it writes the same LDS
  }
}

// Adds the parts of one sequence and query head.  A unit's parts lie with
// consecutive blocks; each of the 256 / (D / 4) rows of threads adds every
// kRows-th of them in order, then the rows are added in order.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p) {
  constexpr int kQuads = D / 4, kRows = 256 / kQuads;
  __shared__ f32x4 lo[kRows][kQuads];
  __shared__ float ll[kRows], lm[4];
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / p.a.q_heads;
  const unsigned hq = (unsigned)(bh % p.a.q_heads), head = hq / p.group, gh = hq % p.group;
  const unsigned unit_heads = p.block_tiles * kHeadTile, units = p.c.heads * p.tile_groups;
  const int d4 = threadIdx.x % kQuads, row = threadIdx.x / kQuads;
  const unsigned begin = p.first[b], n = (p.first[b + 1] - begin) / units;
  if (n == 0) {  // an empty sequence
    if (row == 0) store_out(p.a, bh * D + 4 * d4, (f32x4){0, 0, 0, 0});
    return;
  }
  const unsigned per = range_tiles(p.first[p.a.batch]);
  const unsigned u_first = begin + (head * p.tile_groups + gh / unit_heads) * n;
  const unsigned k0 = u_first / per, k1 = (u_first + n - 1) / per;
  if (k0 == k1) return;  // one block had it all and wrote it
  const unsigned hh = gh % unit_heads;
  // part k of the unit: the block that opened it, then the ones after it
  auto slot = [&](unsigned k) { return (int64_t)(2 * k + (k == k0 ? 1 : 0)) * unit_heads + hh; };
  float top = -INFINITY;
  for (unsigned k = k0 + threadIdx.x; k <= k1; k += 256) top = fmaxf(top, p.part_ml[2 * slot(k)]);
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor(top, m, 64));
  if ((threadIdx.x & 63) == 0) lm[threadIdx.x >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(lm[0], lm[1]), fmaxf(lm[2], lm[3]));
  f32x4 o = {0, 0, 0, 0};
  float sum = 0;
#pragma unroll 4
  for (unsigned k = k0 + row; k <= k1; k += kRows) {
    const int64_t sl = slot(k);
    const float mw = p.part_ml[2 * sl];
    const float f = mw > -INFINITY ? __builtin_amdgcn_exp2f(mw - top) : 0.0f;
    sum += f * p.part_ml[2 * sl + 1];
    o += *(const f32x4*)(p.part_o + sl * D + 4 * d4) * f;
  }
  lo[row][d4] = o;
  if (d4 == 0) ll[row] = sum;
  __syncthreads();
  if (row != 0) return;
#pragma unroll
  for (int r = 1; r < kRows; r++) {
    o += lo[r][d4];
    sum += ll[r];
  }
  store_out(p.a, bh * D + 4 * d4, finish(p.a, hq, top, sum, o));
}

constexpr int kUnitTiles = 16;  // see attend_ranges

}  // namespace

// Head tiles of 16 per cache head; a unit takes up to four.
static int64_t head_tiles(unsigned q_heads, const KvShape& c) { return (q_heads / c.heads + kHeadTile - 1) / kHeadTile; }
static int64_t tile_groups(unsigned q_heads, const KvShape& c) { return (head_tiles(q_heads, c) + kWaves - 1) / kWaves; }
static int64_t unit_tiles16(unsigned q_heads, const KvShape& c) {
  const int64_t t = head_tiles(q_heads, c);
  return t >= 3 ? 4 : t;
}

// Tiles of the longest sequence that the table can name.
static int64_t most_tiles(const KvShape& c, int64_t table_width, int64_t window) {
  int64_t most = std::min<int64_t>(table_width << c.page_shift, kMaxLen);
  if (window > 0 && window < most) most = std::min(most, window + kTile);
  return (most + kTile - 1) / kTile;
}

// Whether blocks take ranges of the flattened tiles; a block takes a unit
// where none is longer than a few tiles, or all are short and there are enough
// of them to fill the chip.
static bool attend_ranges(int64_t units, int64_t tiles) {
  return !(tiles <= kWaves || (tiles <= kUnitTiles && units >= 128));
}

int64_t attend_blocks(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  const int64_t units = batch * c.heads * tile_groups(q_heads, c), tiles = most_tiles(c, table_width, window);
  // flattened tile indexes are 32 bits, with room for one range more
  if (units > (0x7FFFFFFF - 4096) / tiles) return -1;
  if (!attend_ranges(units, tiles)) return units;
  return std::min<int64_t>(1 << kRangeShift, units * ((tiles + kWaves - 1) / kWaves));
}

int64_t attend_workspace(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  if (!attend_ranges(batch * c.heads * tile_groups(q_heads, c), most_tiles(c, table_width, window))) return 0;
  const int64_t blocks = attend_blocks(batch, q_heads, c, table_width, window);
  const int64_t first = ((batch + 1) * 4 + 15) / 16 * 16;
  return first + 2 * blocks * unit_tiles16(q_heads, c) * kHeadTile * (int64_t)(c.dim + 2) * 4;
}

hipError_t launch_attend(const AttendArgs& a, const KvShape& c, bool fp4, void* workspace, hipStream_t st) {
  AttendParams p;
  p.a = a;
  p.c = c;
  p.group = a.q_heads / c.heads;
  p.tiles16 = (unsigned)head_tiles(a.q_heads, c);
  p.tile_groups = (unsigned)tile_groups(a.q_heads, c);
  p.block_tiles = (unsigned)unit_tiles16(a.q_heads, c);
  const int64_t blocks = attend_blocks(a.batch, a.q_heads, c, a.table_width, a.window);
  p.ranges = attend_ranges(a.batch * c.heads * p.tile_groups, most_tiles(c, a.table_width, a.window));
  p.first = (unsigned*)workspace;
  p.part_o = (float*)((uint8_t*)workspace + ((a.batch + 1) * 4 + 15) / 16 * 16);
  p.part_ml = p.part_o + 2 * blocks * p.block_tiles * kHeadTile * c.dim;
  const dim3 grid((unsigned)blocks), block(kThreads);
#define MXQ_ATTEND_T(D, T) fp4 ? k_attend<D, true, T><<<grid, block, 0, st>>>(p) : k_attend<D, false, T><<<grid, block, 0, st>>>(p)
#define MXQ_ATTEND(D)                                                                                  \
  do {                                                                                                 \
    if (a.bf16_out) MXQ_ATTEND_T(D, 2);                                                                \
    else MXQ_ATTEND_T(D, 3);                                                                           \
    if (p.ranges) k_attend_join<D><<<dim3((unsigned)(a.batch * a.q_heads)), dim3(256), 0, st>>>(p);    \
  } while (0)
  if (c.dim == 64) MXQ_ATTEND(64);
  else if (c.dim == 128) MXQ_ATTEND(128);
  else MXQ_ATTEND(256);
#undef MXQ_ATTEND
#undef MXQ_ATTEND_T
  return hipGetLastError();
}

}  // namespace mxq
