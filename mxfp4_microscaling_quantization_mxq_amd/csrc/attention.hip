// attention.hip -- attention of one new token per sequence over a paged
// MXFP8 / MXFP4 cache, split over the cache's length and joined (gfx950).
//
//   o = sum_t p_t V_t / (sum_t p_t [+ exp(sink - m)]),  p_t = exp(scale q . K_t - m),
//   t in [max(0, len - window), len), m the running maximum
//
// Mapping.  The query heads that share a cache head are the 16 columns of the
// 16x16x32 bf16 MFMA (more of them: further waves of the block take further
// groups of 16), and a wave walks over tiles of 32 tokens:
//   S^T = K Q^T: K rows as the A operand, 16 tokens a product.  Lane (i =
//     lane & 15, g = lane >> 4) holds tokens i and 16 + i and 32 consecutive
//     elements 128 p + 32 g of their rows, so a share has one scale, and the
//     results put tokens 4 g + r and 16 + 4 g + r (r < 4) of head i into lane
//     (i, g);
//   O^T += V^T P^T: those eight probabilities ARE the B operand's k slots, so
//     P never crosses lanes.  The A operand is V^T: lane (i, g) loads D / 16
//     consecutive elements of the same eight tokens, and product j takes
//     element j of them (row i <-> d = i D / 16 + j), which turns the
//     transpose of V into byte selects inside the lane.
// Either half of a tile lies in one page, so every address is a scalar base
// (a buffer resource) plus a constant lane offset.  A half that is not there
// (past the length, or a table entry that names no page) has a resource of
// size zero: its loads return zeros and move nothing, so the loop loads
// without branches and the compiler's wait counts leave the tiles ahead in flight.
// Dequantized E4M3 / E2M1 values are exact in bf16.  Scores, maxima, sums and
// O are fp32.  P enters the product as a sum of bf16 terms: two (2^-17 of P)
// for bf16 output, where one term's 2^-9 would add to the output's own
// rounding, and three (2^-25) for fp32 output.
//
// Memory bound: the cache is read once (2 x 1.03 bytes a token, head and
// element in MXFP8, 2 x 0.53 in MXFP4).  64 query heads over 8, D = 128, medians
// of a kernel trace, without the join's 4 to 7 us: 64 sequences of 8192 tokens
// in MXFP8 177 us (6.3 TB/s; 181 with fp32 output), 1 of 131072 47 (5.9), 32 of
// 24000 in MXFP4 159 (5.3; 176).
//
// Split.  A unit is one sequence and one cache head (and up to 64 of its query
// heads); its work is its visible tiles.  The tiles of all units, in order,
// are cut into equal ranges, one a block of 4 waves, so a batch of uneven
// lengths keeps every CU busy to the end.  A range that ends inside a unit
// leaves partial results (m, sum, O) in the workspace, and k_attend_join adds
// a unit's parts in order.  Where all sequences are short, a block takes
// one unit and nothing is joined.
#include "mxq_gemm_common.h"
#include "mxq_kv.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 32;       // tokens a wave takes at a time
constexpr int kWaves = 4;       // waves of a block
constexpr int kThreads = 64 * kWaves;
constexpr int kHeadTile = 16;   // query heads of one MFMA column set
constexpr int64_t kMaxLen = 0x7FFF0000;  // tokens of a sequence (token indexes, also a few tiles past it, are 32 bits)
constexpr float kLog2e = 1.4426950408889634f;

struct AttendParams {
  AttendArgs a;
  KvShape c;
  unsigned group;        // query heads per cache head
  unsigned tile_groups;  // units per sequence and cache head
  unsigned block_tiles;  // head tiles of a unit: 1, 2 or 4
  // Workspace: for each unit that spans blocks, {its parts, the block that
  // opened it, the unit}.  With many units (by_block) the records are indexed
  // by that block (a block opens at most one unit without closing it), else by
  // unit; records with fewer than two parts name nothing to join.
  bool by_block;
  int* parts;               // [blocks or units][4]
  float *part_o, *part_ml;  // [2 blocks][16 block_tiles][D], [2 blocks][16 block_tiles][2]
};

// The compiler keeps what it cannot prove to be the same in every lane in
// vector registers; loop bounds and addresses are scalar only with this.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The arguments of a kernel whose only argument is p.  With kAgain they are read
// again at each call: what only one phase of the kernel uses then occupies no
// scalar register in the others (the tile loop's resources take most of them,
// and scalars that do not fit are kept in vector registers).  The kernels of
// ranges keep 15 such scalars for 57 to 66 without it (their times differ by less
// than two runs of one build do); that of units, which has fewer phases, is 4-29 %
// slower with it (the loop waits for scalar loads it would have kept).
template <bool kAgain>
__device__ __forceinline__ const AttendParams& args(const AttendParams& p) {
  if constexpr (!kAgain) return p;
  uint64_t k = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(k));
  return *(const AttendParams*)(const __attribute__((address_space(4))) AttendParams*)k;
}

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

// Blocks that share the flattened list: as many as keep the memory busy.  Eight
// waves a CU do that with rows of 128 bytes and more; sixteen with rows of 64
// and less, whose tiles are half the bytes for the same instructions.
constexpr int range_shift(int row_bytes) { return row_bytes >= 128 ? 9 : 10; }

// Tiles of a range: an equal share of 2^shift blocks, and enough to give every
// wave one.
__device__ __forceinline__ unsigned range_tiles(unsigned sum, int shift) {
  return max((sum >> shift) + ((sum & ((1u << shift) - 1)) != 0), (unsigned)kWaves);
}

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
template <int D, bool kFp4>
__device__ __forceinline__ void load_k(const AttendParams& p, Half f, int h, int i, int g, Tile<D, kFp4>& t) {
  typedef Tile<D, kFp4> T;
  const __amdgpu_buffer_rsrc_t rq = panel_rsrc(p.a.kq + f.row * T::kRow, f.on ? 16 * T::kRow : 0);
  const __amdgpu_buffer_rsrc_t rs = panel_rsrc(p.a.ks + f.row * (D / 32), f.on ? 16 * (D / 32) : 0);
#pragma unroll
  for (int r = 0; r < T::kRuns; r++) {
    load_bytes<T::kRun>(rq, i * T::kRow + g * T::kRun + r * 4 * T::kRun, t.k[h] + r * T::kRun / 4);
    t.ks[h][r] = __builtin_amdgcn_raw_buffer_load_b8(rs, i * (D / 32) + (D == 64 ? g >> 1 : g + 4 * r), 0, 0);
  }
}
template <int D, bool kFp4>
__device__ __forceinline__ void load_v(const AttendParams& p, Half f, unsigned pos, int h, int i, int g,
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
__device__ __forceinline__ void store_out(const AttendArgs& a, int64_t at, f32x4 o) {
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
__device__ __forceinline__ f32x4 finish(const AttendArgs& a, int64_t hq, float m, float sum, f32x4 o) {
  // Nothing visible.  (Scores that are all NaN leave m there too, and a NaN sum.)
  if (!(m > -INFINITY) && sum == 0) return (f32x4){0, 0, 0, 0};
  if (a.sinks) {
    const float sk = a.sinks[hq] * kLog2e, top = fmaxf(m, sk), f = __builtin_amdgcn_exp2f(m - top);
    sum = sum * f + __builtin_amdgcn_exp2f(sk - top);
    o *= f;
  }
  return o / sum;
}

// Waves a SIMD: what range_shift counts on.  With two or more (at most 256
// registers a wave) the accumulators stay out of the AGPR file, whose moves
// would cost 64 instructions a tile.
template <int D, bool kFp4, int kTerms, bool kRanges>
__global__ __launch_bounds__(kThreads, 1 << (range_shift(kFp4 ? D / 2 : D) - 8)) void k_attend(AttendParams params) {
  typedef Tile<D, kFp4> T;
  constexpr int kRangeShift = range_shift(T::kRow);
  constexpr int kSteps = D / 32;  // QK products of half a tile
  constexpr int J = D / 16;       // PV products of a tile; elements of V per lane and token
  constexpr int kPad = D + 4;
  __shared__ float lds_o[kWaves][kHeadTile][kPad];
  __shared__ float lds_m[kWaves][kHeadTile], lds_l[kWaves][kHeadTile], lds_top[kWaves][kHeadTile];
  __shared__ unsigned lds_sum[kWaves];
  __shared__ int lds_at[5];

  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // This block's tiles: [x, end) of the flattened list, starting in unit
  // (b, head, tile group tg), whose first tile is u_first.
  unsigned x, end, u_first, head, tg, per = 0;
  int64_t b;
  Span s;
  if constexpr (!kRanges) {
    const AttendParams& p = args<kRanges>(params);
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
    const AttendParams& p = args<kRanges>(params);
    // each thread sums the tiles of a run of sequences; scan over the block
    const unsigned units = p.c.heads * p.tile_groups;  // of a sequence
    const unsigned batch = (unsigned)p.a.batch, each = (batch + kThreads - 1) / kThreads;
    const unsigned b0 = min(threadIdx.x * each, batch), b1 = min(b0 + each, batch);
    unsigned own = 0;
    bool empty = false;  // a sequence of this thread's run has no tiles
    for (unsigned k = b0; k < b1; k++) {
      s = span_of(p, k);
      own += (s.t1 - s.t0) * units;
      empty |= s.t0 == s.t1;
    }
    unsigned incl = own;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const unsigned o = __shfl_up(incl, m, 64);
      if (lane >= m) incl += o;
    }
    if (lane == 63) lds_sum[wave] = incl;
    const bool any_empty = __syncthreads_or(empty);
    unsigned sum = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      if (w < wave) before += lds_sum[w];
      sum += lds_sum[w];
    }
    sum = uniform(sum);
    per = range_tiles(sum, kRangeShift);
    x = blockIdx.x * per;
    end = min(x + per, sum);
    unsigned at = before + incl - own;  // first tile of this thread's sequences
    if (x >= at && x < at + own) {
      unsigned k = b0;
      if (each > 1) {  // (a run of one sequence: s is its span)
        s = span_of(p, k);
        while (x >= at + (s.t1 - s.t0) * units) {
          at += (s.t1 - s.t0) * units;
          s = span_of(p, ++k);
        }
      }
      const unsigned n = s.t1 - s.t0, u = (x - at) / n;
      lds_at[0] = (int)k, lds_at[1] = (int)u, lds_at[2] = (int)(at + u * n), lds_at[3] = s.start, lds_at[4] = s.len;
    }
    // the zeros of empty sequences, each by one block
    for (unsigned k = any_empty ? blockIdx.x : batch; k < batch; k += gridDim.x) {
      s = span_of(p, k);
      if (s.t0 != s.t1) continue;
      for (unsigned e = threadIdx.x; e < p.a.q_heads * (D / 4); e += kThreads)
        store_out(p.a, (int64_t)k * p.a.q_heads * D + 4 * e, (f32x4){0, 0, 0, 0});
      if (!p.by_block)
        for (unsigned u = threadIdx.x; u < units; u += kThreads) p.parts[4 * (k * units + u)] = 0;
    }
    if (p.by_block && threadIdx.x == 0) p.parts[4 * blockIdx.x] = 0;
    if (x >= end) return;
    __syncthreads();
    b = uniform(lds_at[0]);
    const unsigned u = uniform(lds_at[1]);
    u_first = uniform(lds_at[2]);
    s = span_tiles(uniform(lds_at[3]), uniform(lds_at[4]));
    head = u, tg = 0;
    if (p.tile_groups > 1) head = u / p.tile_groups, tg = u % p.tile_groups;
  }

  // waves per head tile (a power of two), and this wave among them
  const unsigned block_tiles = args<kRanges>(params).block_tiles;
  const unsigned per_shift = block_tiles == 4 ? 0 : block_tiles == 2 ? 1 : 2;
  const unsigned per_tile = 1u << per_shift;
  const int sub = wave & (per_tile - 1);
  const unsigned wave_h0 = (wave >> per_shift) * kHeadTile;

  while (true) {
    // tiles [first, last) of the unit
    s = span_tiles(uniform(s.start), uniform(s.len));
    x = uniform(x), end = uniform(end), u_first = uniform(u_first), head = uniform(head), tg = uniform(tg);
    b = uniform((int)b);
    const int first = s.t0 + (int)(x - u_first), last = min(s.t1, s.t0 + (int)(end - u_first));
    unsigned h0;  // first query head of the unit

    // of the unscaled scores, and of this lane's tokens
    float m = -INFINITY, l = 0, to_log2;
    f32x4 acc[J];
#pragma unroll
    for (int j = 0; j < J; j++) acc[j] = (f32x4){0, 0, 0, 0};
    {
      const AttendParams& p = args<kRanges>(params);
      h0 = tg * p.block_tiles * kHeadTile;
      const unsigned shift = p.c.page_shift, pmask = (1u << shift) - 1;
      // scores are scaled by |scale| (its sign is in q), never by less than what
      // keeps a masked score at -inf
      to_log2 = fmaxf(fabsf(p.a.scale) * kLog2e, 0x1p-100f);
      const unsigned q_sign = p.a.scale < 0 ? 0x80008000u : 0u;

      // Q^T as the B operand: lane (i, g) holds the elements of head i that pair
      // with the K elements of lane group g
      const unsigned gh = h0 + wave_h0 + i;
      const bool live = h0 + wave_h0 < p.group;
      bf16x8 qf[kSteps];
#pragma unroll
      for (int st = 0; st < kSteps; st++) {
        const int d = D == 64 ? 16 * g + 8 * st : 128 * (st / 4) + 32 * g + 8 * (st & 3);
        u32x4 w = {0, 0, 0, 0};
        if (gh < p.group) w = *(const u32x4*)(p.a.q + b * p.a.q_stride + (int64_t)(head * p.group + gh) * D + d);
        qf[st] = __builtin_bit_cast(bf16x8, w ^ q_sign);
      }

      // This wave's tiles are first + sub + per_tile j, j < count.  The page ids
      // of the tile to load next are scalars, read from the table one tile
      // earlier; -1 where the table names no page of the cache.
      const __attribute__((address_space(4))) int32_t* row =
          (const __attribute__((address_space(4))) int32_t*)(p.a.table + b * p.a.table_stride);
      const int count = live && first + sub < last ? (last - first - sub + (int)per_tile - 1) >> per_shift : 0;
      auto token_of = [&](int j) { return (first + sub + (j << per_shift)) * kTile; };
      auto id_of = [&](int token) { return uniform(row[(unsigned)min(token, s.len - 1) >> shift]); };
      int id0 = id_of(token_of(0)), id1 = id_of(token_of(0) + 16);
      int fetched = 0;  // tiles whose K is on its way

      T t;
      Half half[2];  // of the tile in t
      auto fetch_k = [&]() {
        const int tok = token_of(fetched);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int id = h ? id1 : id0, th = tok + 16 * h;
          half[h].on = fetched < count && th < s.len && id >= 0 && id < p.c.pages;
          half[h].row = (((int64_t)(half[h].on ? id : 0) * p.c.heads + head) << shift) + (th & pmask);
          load_k<D, kFp4>(p, half[h], h, i, g, t);
        }
        fetched++;
        const int next = token_of(min(fetched, count - 1));
        id0 = id_of(next);
        id1 = id_of(next + 16);
      };
      auto fetch_v = [&](int j) {
#pragma unroll
        for (int h = 0; h < 2; h++) load_v<D, kFp4>(p, half[h], (token_of(j) + 16 * h) & pmask, h, i, g, t);
      };
      if (count > 0) {
        fetch_k();
        fetch_v(0);
      }
      for (int j = 0; j < count; j++) {
        const int t0 = token_of(j);
        const bool on0 = half[0].on, on1 = half[1].on;
        // S^T
        f32x4 sc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int st = 0; st < kSteps; st++)
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const float scale = e8m0_as_scale(t.ks[h][D == 64 ? 0 : st / 4]);
            u32x4 a;
#pragma unroll
            for (int e = 0; e < 4; e++) a[e] = decode2<kFp4>(t.k[h], 4 * st + e, scale);
            sc[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), qf[st], sc[h], 0, 0, 0);
          }
        fetch_k();
        // softmax over the tile; y[4 h + r]: head i, token t0 + 16 h + 4 g + r
        float y[8];
#pragma unroll
        for (int r = 0; r < 8; r++) y[r] = sc[r >> 2][r & 3];
        const bool whole = t0 >= s.start && t0 + kTile <= s.len && on0 && on1;
        if (!whole) {
          // a masked token's K and V bytes are whatever the page holds: its
          // score is replaced, and its codes and scale are cleared, so nothing
          // of it (NaN codes among it) reaches a product with a non-zero factor
#pragma unroll
          for (int r = 0; r < 8; r++) {
            const int tok = t0 + 16 * (r >> 2) + 4 * g + (r & 3);
            const bool seen = (r < 4 ? on0 : on1) && tok >= s.start && tok < s.len;
            y[r] = seen ? y[r] : -INFINITY;
#pragma unroll
            for (int w = 0; w < (int)(sizeof(t.v[r]) / 4); w++) t.v[r][w] = seen ? t.v[r][w] : 0u;
            t.vs[r >> 2] = seen ? t.vs[r >> 2] : t.vs[r >> 2] & ~(0xFFu << (8 * (r & 3)));
          }
        }
        float top = y[0];
#pragma unroll
        for (int r = 1; r < 8; r++) top = fmaxf(top, y[r]);
        top = fmaxf(m, max_groups(top));
        const float ref = top > -INFINITY ? top * to_log2 : 0.0f;  // nothing seen yet: every p is 0
        if (__builtin_amdgcn_ballot_w64(top > m) != 0) {
          // the old terms are relative to the rounded m * to_log2, so that is what
          // moves them: exactly 1 for a head whose maximum stays
          const float alpha = __builtin_amdgcn_exp2f(m * to_log2 - ref);
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
        for (int r = 0; r < 8; r++) vscale[r] = e8m0_as_scale((t.vs[r >> 2] >> (8 * (r & 3))) & 0xFFu);
#pragma unroll
        for (int j2 = 0; j2 < J / 2; j2++) {
          unsigned d[8];
#pragma unroll
          for (int r = 0; r < 8; r++) d[r] = decode2<kFp4>(t.v[r], j2, vscale[r]);
          u32x4 va[2];
#pragma unroll
          for (int r = 0; r < 4; r++) {
            va[0][r] = perm(d[2 * r + 1], d[2 * r], 0x05040100u);
            va[1][r] = perm(d[2 * r + 1], d[2 * r], 0x07060302u);
          }
#pragma unroll
          for (int k = 0; k < kTerms; k++)
#pragma unroll
            for (int o = 0; o < 2; o++)
              acc[2 * j2 + o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, va[o]), __builtin_bit_cast(bf16x8, pt[k]), acc[2 * j2 + o], 0, 0, 0);
        }
        fetch_v(j + 1);
      }
    }

    // join the waves of a head tile (maxima in log2 units from here on)
    const AttendParams& p = args<kRanges>(params);
    l = sum_groups(l);
    m *= to_log2;
    if (g == 0) lds_m[wave][i] = m;
    __syncthreads();
    float mt = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
      const float mw = lds_m[w][i];
      mt = w >> per_shift == wave >> per_shift ? fmaxf(mt, mw) : mt;
    }
    const float f = m > -INFINITY ? __builtin_amdgcn_exp2f(m - mt) : 0.0f;
    if (g == 0) lds_l[wave][i] = l * f;
    if (g == 0 && sub == 0) lds_top[wave][i] = mt;
#pragma unroll
    for (int j = 0; j < J; j++)
#pragma unroll
      for (int r = 0; r < 4; r++) lds_o[wave][i][(4 * g + r) * J + j] = acc[j][r] * f;
    __syncthreads();

    // out: threads over (head of the unit, 4 elements)
    constexpr int kQuads = D / 4;
    const bool opens = first == s.t0, closes = last == s.t1;  // of the unit
    if (kRanges && opens && threadIdx.x == 0 && !(p.by_block && closes)) {
      const unsigned unit = ((unsigned)b * p.c.heads + head) * p.tile_groups + tg;
      int* w = p.parts + 4 * (p.by_block ? blockIdx.x : unit);
      w[0] = (int)((u_first + (unsigned)(s.t1 - s.t0) - 1) / per - blockIdx.x) + 1;
      w[1] = (int)blockIdx.x, w[2] = (int)unit;
    }
    const unsigned heads = min(p.group - h0, p.block_tiles * kHeadTile);
    for (unsigned e = threadIdx.x; e < heads * kQuads; e += kThreads) {
      const unsigned hh = e / kQuads, d4 = e % kQuads;
      const unsigned wb = hh / kHeadTile << per_shift;
      const float mx = lds_top[wb][hh % kHeadTile];
      float sum = 0;
      f32x4 o = {0, 0, 0, 0};
#pragma unroll
      for (unsigned w = 0; w < kWaves; w++) {
        if (w >= per_tile) break;
        sum += lds_l[wb + w][hh % kHeadTile];
        o += *(const f32x4*)&lds_o[wb + w][hh % kHeadTile][4 * d4];
      }
      if (!kRanges || (opens && closes)) {
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
    if constexpr (!kRanges) break;
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

// Adds the parts of the unit of record blockIdx.x: slot 1 of the block that
// opened it, then slot 0 of the blocks after it.  A block takes kHeads heads
// (grid y), with kRows rows of D / 4 threads each; a row adds every kRows-th
// part in order, then the rows are added in order.
template <int D, int kHeads>
__global__ __launch_bounds__(256) void k_attend_join(AttendParams p) {
  constexpr int kQuads = D / 4, kRows = 256 / kQuads / kHeads;
  __shared__ f32x4 lo[256 / kQuads][kQuads];
  __shared__ float ll[256 / kQuads], lm[256 / kQuads];
  const int* w = p.parts + 4 * blockIdx.x;
  const int parts = w[0];
  if (parts < 2) return;
  const unsigned k0 = w[1], unit = w[2];
  const unsigned unit_heads = p.block_tiles * kHeadTile;
  const unsigned h0 = unit % p.tile_groups * unit_heads, head = unit / p.tile_groups % p.c.heads;
  const int64_t b = unit / (p.tile_groups * p.c.heads);
  const int d4 = threadIdx.x % kQuads, line = threadIdx.x / kQuads, row = line % kRows;
  const unsigned hh = blockIdx.y * kHeads + line / kRows;
  const bool live = hh < unit_heads && h0 + hh < p.group;
  auto slot = [&](int part) { return (int64_t)(2 * (k0 + part) + (part == 0 ? 1 : 0)) * unit_heads + hh; };
  float top = -INFINITY, sum = 0;
  f32x4 o = {0, 0, 0, 0};
  if (live) {
    // a row's parts four at a time, all loads first
    constexpr int kN = 4;
    for (int k = row; k < parts; k += kN * kRows) {
      f32x2 ml[kN];
      f32x4 po[kN];
#pragma unroll
      for (int c = 0; c < kN; c++) {
        const int64_t sl = slot(min(k + c * kRows, parts - 1));
        ml[c] = *(const f32x2*)(p.part_ml + 2 * sl);
        po[c] = *(const f32x4*)(p.part_o + sl * D + 4 * d4);
      }
      float m = top;
#pragma unroll
      for (int c = 0; c < kN; c++) m = fmaxf(m, ml[c].x);
      const float ref = m > -INFINITY ? m : 0.0f, f0 = __builtin_amdgcn_exp2f(top - ref);
      sum *= f0;
      o *= f0;
      top = m;
#pragma unroll
      for (int c = 0; c < kN; c++) {
        const float f = k + c * kRows < parts ? __builtin_amdgcn_exp2f(ml[c].x - ref) : 0.0f;
        sum += f * ml[c].y;
        o += po[c] * f;
      }
    }
  }
  if constexpr (kRows > 1) {
    lo[line][d4] = o;
    if (d4 == 0) ll[line] = sum, lm[line] = top;
    __syncthreads();
    if (row != 0) return;
#pragma unroll
    for (int r = 1; r < kRows; r++) top = fmaxf(top, lm[line + r]);
    const float ref = top > -INFINITY ? top : 0.0f;
    o = (f32x4){0, 0, 0, 0};
    sum = 0;
#pragma unroll
    for (int r = 0; r < kRows; r++) {
      const float f = __builtin_amdgcn_exp2f(lm[line + r] - ref);
      o += lo[line + r][d4] * f;
      sum += ll[line + r] * f;
    }
  }
  if (!live) return;
  const int64_t hq = (int64_t)head * p.group + h0 + hh;
  store_out(p.a, (b * p.a.q_heads + hq) * D + 4 * d4, finish(p.a, hq, top, sum, o));
}

}  // namespace

// Head tiles of 16 per cache head; a unit takes up to four.
static int64_t head_tiles(unsigned q_heads, const KvShape& c) {
  return (q_heads / c.heads + kHeadTile - 1) / kHeadTile;
}
static int64_t tile_groups(unsigned q_heads, const KvShape& c) {
  return (head_tiles(q_heads, c) + kWaves - 1) / kWaves;
}
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

// Whether blocks take ranges of the flattened tiles: where a unit would keep
// one block longer than the join of its parts takes, which is a second launch
// (4 us of GPU time and 4 us of the host's).  A block needs about 1 us for 4
// tiles, and the more units there are, the longer the others take anyway.  64
// query heads over 8, D = 128, MXFP8, ranges / units in a graph's replays: 1
// sequence of 500 tokens (16 tiles, 8 units) 9.2 / 7.7 us, of 1000 9.7 / 11.8
// (but two launches); 8 of 700-1000 (32 tiles, 64 units) 15.5 / 11.8; 16 of
// 1500-2000 (63 tiles, 128 units) 23.0 / 21.4, 64 53.5 / 45.7; 16 of 1000-4000
// 27.1 / 35.4, 64 72 / 75; D = 64, 97 of 0-3999 with a window of 128 16.5 / 8.7,
// in MXFP4 16.3 / 8.3.
static bool attend_ranges(int64_t units, int64_t tiles) { return tiles > (units >= 128 ? 64 : 32); }

int64_t attend_blocks(int64_t batch, unsigned q_heads, const KvShape& c, bool fp4, int64_t table_width,
                      int64_t window) {
  const int64_t units = batch * c.heads * tile_groups(q_heads, c), tiles = most_tiles(c, table_width, window);
  // flattened tile indexes are 32 bits, with room for one range more
  if (units > (0x7FFFFFFF - 4096) / tiles) return -1;
  if (!attend_ranges(units, tiles)) return units;
  return std::min<int64_t>(1 << range_shift(fp4 ? c.dim / 2 : c.dim), units * ((tiles + kWaves - 1) / kWaves));
}

int64_t attend_workspace(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window) {
  if (!attend_ranges(batch * c.heads * tile_groups(q_heads, c), most_tiles(c, table_width, window))) return 0;
  // for either format: the smaller rows take no fewer blocks (nor records)
  const int64_t blocks = attend_blocks(batch, q_heads, c, true, table_width, window);
  return blocks * (16 + 2 * unit_tiles16(q_heads, c) * kHeadTile * (int64_t)(c.dim + 2) * 4);
}

// With a range for each unit or so (by_block), a unit has two or three parts,
// which one row of threads adds; with fewer units they have many, and the rows
// of a block share them.
template <int D>
static void launch_join(const AttendParams& p, unsigned heads, int64_t records, hipStream_t st) {
  constexpr int kLines = 256 / (D / 4), kFew = kLines > 8 ? kLines / 8 : 1;
  if (p.by_block)
    k_attend_join<D, kLines><<<dim3((unsigned)records, (heads + kLines - 1) / kLines), dim3(256), 0, st>>>(p);
  else
    k_attend_join<D, kFew><<<dim3((unsigned)records, (heads + kFew - 1) / kFew), dim3(256), 0, st>>>(p);
}

hipError_t launch_attend(const AttendArgs& a, const KvShape& c, bool fp4, void* workspace, hipStream_t st) {
  AttendParams p;
  p.a = a;
  p.c = c;
  p.group = a.q_heads / c.heads;
  p.tile_groups = (unsigned)tile_groups(a.q_heads, c);
  p.block_tiles = (unsigned)unit_tiles16(a.q_heads, c);
  const int64_t blocks = attend_blocks(a.batch, a.q_heads, c, fp4, a.table_width, a.window);
  const int64_t units = a.batch * c.heads * p.tile_groups;
  const bool ranges = attend_ranges(units, most_tiles(c, a.table_width, a.window));
  p.by_block = units >= blocks / 2;
  p.parts = (int*)workspace;  // at most a record a block, in either case
  p.part_o = (float*)((uint8_t*)workspace + blocks * 16);
  p.part_ml = p.part_o + 2 * blocks * p.block_tiles * kHeadTile * c.dim;
  const dim3 grid((unsigned)blocks), block(kThreads);
  const unsigned heads = std::min(p.group, p.block_tiles * kHeadTile);
#define MXQ_ATTEND_R(D, F, T) \
  ranges ? k_attend<D, F, T, true><<<grid, block, 0, st>>>(p) : k_attend<D, F, T, false><<<grid, block, 0, st>>>(p)
#define MXQ_ATTEND(D)                                                                              \
  do {                                                                                             \
    if (a.bf16_out && fp4) MXQ_ATTEND_R(D, true, 2);                                               \
    else if (a.bf16_out) MXQ_ATTEND_R(D, false, 2);                                                \
    else if (fp4) MXQ_ATTEND_R(D, true, 3);                                                        \
    else MXQ_ATTEND_R(D, false, 3);                                                                \
    if (ranges) launch_join<D>(p, heads, p.by_block ? blocks : units, st);                         \
  } while (0)
  if (c.dim == 64) MXQ_ATTEND(64);
  else if (c.dim == 128) MXQ_ATTEND(128);
  else MXQ_ATTEND(256);
#undef MXQ_ATTEND
#undef MXQ_ATTEND_R
  return hipGetLastError();
}

}  // namespace mxq
