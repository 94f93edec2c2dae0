// tree_attention.hip -- attention of several drafted tokens per sequence over a
// paged MXFP8 / MXFP4 cache, each of which sees the context and the drafted
// tokens that its mask names (gfx950).
//
//   o_i = sum_t p_t V_t / (sum_t p_t [+ exp(sink - m)]),  p_t = exp(scale q_i . K_t - m),
//   t over the context and over context + j for the bits j of mask i
//
// Rows.  The query heads that share a cache head, of all drafted tokens, are the
// rows of one product with the cache: row r is head r % group of token r / group.
// A wave takes N sets of 16 rows (the columns of the 16x16x32 bf16 MFMA) and
// walks over tiles of 32 tokens as the attention of one token does: S^T = K Q^T,
// whose results are the B operand of O^T += V^T P^T without leaving their lanes,
// with the transpose of V as byte selects.  A tile is loaded and decoded once for
// the wave's sets.
//
// Masks.  A tile that some row of the wave does not see whole (the context's
// end, a window's edge, the drafted tokens) forms a word of 32 bits a row, from
// two ranges and the row's mask in LDS; all others have no mask at all.
//
// Split.  As for one token: a unit is one sequence, one cache head and a group
// of its rows; the tiles of all units in order are cut into equal ranges, one a
// block, and ranges that end inside a unit leave partial results to be joined.
// Short calls and single sequences are cut by shares instead (tree_plan).
//
// What bounds it.  Few rows: the cache's bytes (64 sequences of 8192 tokens, 8
// query heads over each of 8 cache heads, D = 128, E4M3: 178 us, 6.2 TB/s).  64
// rows: decoding, once for each 32 (64 sequences of 4600 tokens with 8 drafted
// ones 212 us, 2.9 TB/s).  Many rows: products, with P in two bf16 terms or three,
// and the exponentials and the decoding, which a wave does one after another (64
// drafted tokens over 4 x 20500: 322 us, 536 TFLOP/s counted once, 800 as issued; over
// 4 x 9000 to 32000 the matrix cores are busy for 39 % of the time, the vector units
// for 40 %, LDS for 29 %, with two waves a SIMD).
#include "mxq_attend.h"

namespace mxq {

namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kSet = 16;            // rows of one MFMA column set
constexpr int kMaskRow = 2 * 4 + 2;  // 32-bit words of a token's mask in LDS, an empty one before and after

struct TreeParams {
  TreeArgs a;
  KvShape c;
  unsigned group;       // query heads per cache head
  unsigned rows;        // group * drafts
  unsigned row_groups;  // units per sequence and cache head
  unsigned row_shift;   // 2^row_shift waves of a block take rows of their own, the others tiles (k_tree_attend)
  // Workspace, as for one token: records {parts, the block that opened the
  // unit, the unit} by opening block (by_block) or by unit, and two slots of
  // partial results a block.
  bool by_block, split;  // split: blocks take ranges (k_tree_wide; else units)
  unsigned shares;       // equal shares of a unit that a block each takes (where they take no ranges)
  int* parts;
  float *part_o, *part_ml;
};

// What a sequence's rows may see: tiles [0, a) and [b, b + n - a) of kT tokens.
struct TreeSpan {
  int context, end, a, b, n;
};
template <int kT>
__device__ __forceinline__ TreeSpan tree_span(const TreeParams& p, int64_t seq) {
  const int64_t most = min(p.a.table_width << p.c.page_shift, kMaxLen);
  const int64_t context = min((int64_t)max(p.a.context[seq], 0), most), end = min(context + p.a.drafts, most);
  TreeSpan s = {(int)context, (int)end, 0, 0, 0};
  if (p.a.window > 0) {
    s.a = (int)((min(p.a.first, end) + kT - 1) / kT);
    s.b = max(s.a, (int)(max((int64_t)0, context - p.a.window + 1) / kT));
  }
  const int tiles = (int)((end + kT - 1) / kT);
  s.n = s.a + max(0, tiles - s.b);
  if (s.n == 0) s.b = tiles - 1, s.n = 1;  // nothing to see: a tile that is masked, for the zeros
  return s;
}

__device__ __forceinline__ unsigned below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// Context tokens from here on are inside the window of a row of this depth.
__device__ __forceinline__ int window_start(const TreeParams& p, int context, int depth) {
  return (int)max((int64_t)0, context + depth - p.a.window + 1);
}
// Tokens t0 .. t0 + 31 that are seen: of the context those from lo on and the
// first ones, of the drafted ones those of the mask (in LDS, as load_masks lays it out).
__device__ __forceinline__ unsigned seen_word(const TreeSpan& s, int t0, int lo, int seen_first, const unsigned* mask, int words) {
  const int to = s.context - t0;
  unsigned w = (below(to) & ~below(lo - t0)) | below(seen_first - t0);
  const int at = (-to) >> 5;  // drafted token -to is the word's first
  if (at >= -1 && at <= 2 * words - 1) {
    const unsigned* m = mask + 1 + at;
    w |= (unsigned)((((uint64_t)m[1] << 32) | m[0]) >> ((unsigned)-to & 31u));
  }
  return w;
}

// Into LDS: the masks of `tokens` drafted tokens from token0 on, less what the
// window hides, each between two empty words; all of them together (any); all
// tokens' depths; and the largest and smallest depth (far, preset) of these.
__device__ __forceinline__ void load_masks(const TreeParams& p, int64_t b, const TreeSpan& s, unsigned token0, unsigned tokens,
                                           unsigned (*mask)[kMaskRow], unsigned* any, int* depths, int* far) {
  const unsigned words = p.a.words, drafts = (unsigned)p.a.drafts;
  if (threadIdx.x < drafts) {
    const uint32_t* m = (const uint32_t*)(p.a.mask + (b * drafts + threadIdx.x) * words);
    int depth = 0;
    for (unsigned w = 0; w <= threadIdx.x / 32; w++) depth += __popc(m[w] & below((int)(threadIdx.x - 32 * w)));
    depths[threadIdx.x] = depth;
  }
  if (threadIdx.x < kMaskRow) any[threadIdx.x] = 0;
  __syncthreads();
  for (unsigned e = threadIdx.x; e < tokens * 2 * words; e += blockDim.x) {
    const unsigned t = e / (2 * words), w = e - t * 2 * words;
    const int depth = depths[token0 + t];
    unsigned v = ((const uint32_t*)(p.a.mask + (b * drafts + token0 + t) * words))[w] & below((int)drafts - (int)(32 * w));
    if (p.a.window > 0 && p.a.window < p.a.drafts) {
      unsigned left = v;
      while (left) {
        const int bit = __builtin_ctz(left), d = depths[32 * w + bit];
        left &= left - 1;
        if (depth - d >= p.a.window && s.context + d >= p.a.first) v &= ~(1u << bit);
      }
    }
    mask[t][1 + w] = v;
    atomicOr(&any[1 + w], v);
    if (w != 0) continue;
    atomicMax(&far[0], depth);
    atomicMin(&far[1], depth);
    mask[t][0] = mask[t][1 + 2 * words] = 0;
  }
  __syncthreads();
}

// A block's range of the flattened tiles of kT tokens: [x, end), in the unit (b,
// head, rg) whose first tile is u_first; `per` tiles a range, at least `least`.
struct RangeStart {
  unsigned x, end, u_first, head, rg, per;
  int64_t b;
};
template <int kT>
__device__ __forceinline__ RangeStart range_start(const TreeParams& p, unsigned least, unsigned* lds_sum, int* lds_at) {
  // each of 256 threads sums the tiles of a run of sequences; scan over the block
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned units = p.c.heads * p.row_groups;  // of a sequence
  const unsigned batch = (unsigned)p.a.batch, each = (batch + kThreads - 1) / kThreads;
  const unsigned b0 = min(threadIdx.x * each, batch), b1 = min(b0 + each, batch);
  unsigned own = 0;
  for (unsigned k = b0; k < b1; k++) own += tree_span<kT>(p, k).n * units;
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
  RangeStart r;
  sum = uniform(sum);
  r.per = max((sum + gridDim.x - 1) / gridDim.x, least);
  r.x = blockIdx.x * r.per;
  r.end = min(r.x + r.per, sum);
  unsigned at = before + incl - own;  // first tile of this thread's sequences
  if (r.x >= at && r.x < at + own) {
    unsigned k = b0, n = tree_span<kT>(p, k).n;
    while (r.x >= at + n * units) {
      at += n * units;
      n = tree_span<kT>(p, ++k).n;
    }
    const unsigned u = (r.x - at) / n;
    lds_at[0] = (int)k, lds_at[1] = (int)u, lds_at[2] = (int)(at + u * n);
  }
  if (p.by_block && threadIdx.x == 0) p.parts[4 * blockIdx.x] = 0;
  __syncthreads();
  r.b = uniform(lds_at[0]);
  const unsigned u = uniform(lds_at[1]);
  r.u_first = uniform(lds_at[2]);
  r.head = u / p.row_groups, r.rg = u % p.row_groups;
  return r;
}

// Largest value and sum over the two halves of a wave, in every lane.
__device__ __forceinline__ float max_halves(float v) {
  const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
}

template <int D, bool kFp4, int kTerms, int N, bool kRanges>
__global__ __launch_bounds__(kThreads, 2) void k_tree_attend(TreeParams p) {
  typedef Tile<D, kFp4> T;
  constexpr int kSteps = D / 32;  // QK products of half a tile
  constexpr int J = D / 16;       // PV products of a tile; elements of V per lane and token
  constexpr int kPad = D + 4;
  __shared__ float lds_o[kWaves][kSet][kPad];
  __shared__ float lds_m[kWaves][kSet], lds_l[kWaves][kSet], lds_top[kWaves][kSet];
  __shared__ unsigned lds_mask[2 * N * kSet][kMaskRow];
  __shared__ unsigned lds_any[kMaskRow];
  __shared__ int lds_depth[kThreads], lds_far[2];
  __shared__ unsigned lds_sum[kWaves];
  __shared__ int lds_at[3];

  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned per_shift = 2 - p.row_shift, per_tile = 1u << per_shift;  // waves that share tiles
  const int sub = wave & (per_tile - 1), row_wave = wave >> per_shift;
  const unsigned unit_rows = (unsigned)(N * kSet) << p.row_shift;

  unsigned x, end, u_first, head, rg, per = 0;
  int64_t b;
  TreeSpan s;
  if constexpr (!kRanges) {
    unsigned id = blockIdx.x;
    const unsigned share = uniform(id % p.shares);
    id /= p.shares;
    rg = uniform(id % p.row_groups);
    id /= p.row_groups;
    head = uniform(id % p.c.heads);
    b = uniform(id / p.c.heads);
    s = tree_span<kTile>(p, b);
    u_first = 0;
    x = (unsigned)((uint64_t)s.n * share / p.shares);
    end = (unsigned)((uint64_t)s.n * (share + 1) / p.shares);
  } else {
    const RangeStart r = range_start<kTile>(p, per_tile, lds_sum, lds_at);
    if (r.x >= r.end) return;
    x = uniform(r.x), end = uniform(r.end), u_first = uniform(r.u_first), head = uniform(r.head), rg = uniform(r.rg), per = uniform(r.per), b = r.b;
    s = tree_span<kTile>(p, b);
  }

  while (true) {
    // tiles [first, last) of the unit, counted from its first
    const int first = (int)(x - u_first), last = min(s.n, (int)(end - u_first));
    const unsigned row0 = rg * unit_rows, token0 = row0 / p.group;
    const unsigned tokens = (min(row0 + unit_rows, p.rows) - 1) / p.group - token0 + 1;
    const unsigned drafts = (unsigned)p.a.drafts;
    if (threadIdx.x < 2) lds_far[threadIdx.x] = threadIdx.x ? 0x7FFFFFFF : 0;

    // rows: scores are scaled by |scale| (its sign is in q), never by less than
    // what keeps a masked score at -inf
    const float to_log2 = fmaxf(fabsf(p.a.scale) * kLog2e, 0x1p-100f);
    const unsigned q_sign = p.a.scale < 0 ? 0x80008000u : 0u;
    float m[N], l[N];  // of the unscaled scores, and of this lane's tokens
    f32x4 acc[N][J];
    bf16x8 qf[N][kSteps];
    unsigned mask_at[N];
    bool live[N];
#pragma unroll
    for (int n = 0; n < N; n++) {
      m[n] = -INFINITY, l[n] = 0;
#pragma unroll
      for (int j = 0; j < J; j++) acc[n][j] = (f32x4){0, 0, 0, 0};
      const unsigned r = row0 + (row_wave * N + n) * kSet + i;
      live[n] = r < p.rows;
      const unsigned token = live[n] ? r / p.group : token0, qh = head * p.group + (live[n] ? r - token * p.group : 0);
      mask_at[n] = token - token0;
#pragma unroll
      for (int st = 0; st < kSteps; st++) {
        const int d = D == 64 ? 16 * g + 8 * st : 128 * (st / 4) + 32 * g + 8 * (st & 3);
        u32x4 w = {0, 0, 0, 0};
        if (live[n]) w = *(const u32x4*)(p.a.q + (b * drafts + token) * p.a.q_stride + (int64_t)qh * D + d);
        qf[n][st] = __builtin_bit_cast(bf16x8, w ^ q_sign);
      }
    }
    {
      const unsigned shift = p.c.page_shift, pmask = (1u << shift) - 1;
      // This wave's tiles are first + sub + per_tile j, j < count.  The page ids
      // of the tile to load next are scalars, read from the table one tile
      // earlier; -1 where the table names no page of the cache.
      const __attribute__((address_space(4))) int32_t* row =
          (const __attribute__((address_space(4))) int32_t*)(p.a.table + b * p.a.table_stride);
      const bool any_row = row0 + row_wave * N * kSet < p.rows;
      const int count = any_row && first + sub < last ? (last - first - sub + (int)per_tile - 1) >> per_shift : 0;
      auto token_of = [&](int j) {
        const int k = first + sub + (j << per_shift);
        return (k < s.a ? k : k - s.a + s.b) * kTile;
      };
      auto id_of = [&](int token) { return uniform(row[(unsigned)min(token, s.end - 1) >> shift]); };
      int id0 = -1, id1 = -1, fetched = 0;  // tiles whose K is on its way

      T t;
      Half half[2];  // of the tile in t
      auto fetch_k = [&]() {
        const int tok = token_of(fetched);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int id = h ? id1 : id0, th = tok + 16 * h;
          half[h].on = fetched < count && th < s.end && id >= 0 && id < p.c.pages;
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
        id0 = id_of(token_of(0));
        id1 = id_of(token_of(0) + 16);
        fetch_k();
        fetch_v(0);
      }
      // (the masks while the first tile is on its way)
      load_masks(p, b, s, token0, tokens, lds_mask, lds_any, lds_depth, lds_far);
      int lo[N], lo_most = 0;  // context tokens from here on are inside the row's window
#pragma unroll
      for (int n = 0; n < N; n++) {
        lo[n] = p.a.window > 0 ? window_start(p, s.context, lds_depth[token0 + mask_at[n]]) : 0;
        lo_most = live[n] ? max(lo_most, lo[n]) : lo_most;
      }
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) lo_most = max(lo_most, __shfl_xor(lo_most, k, 64));
      lo_most = uniform(lo_most);
      const int seen_first = p.a.window > 0 ? (int)min(p.a.first, (int64_t)s.context) : 0;
      for (int j = 0; j < count; j++) {
        const int t0 = token_of(j);
        const bool on0 = half[0].on, on1 = half[1].on;
        // S^T
        f32x4 sc[N][2];
#pragma unroll
        for (int n = 0; n < N; n++) sc[n][0] = sc[n][1] = (f32x4){0, 0, 0, 0};
#pragma unroll
        for (int st = 0; st < kSteps; st++)
#pragma unroll
          for (int h = 0; h < 2; h++) {
            const float scale = e8m0_as_scale(t.ks[h][D == 64 ? 0 : st / 4]);
            u32x4 a;
#pragma unroll
            for (int e = 0; e < 4; e++) a[e] = decode2<kFp4>(t.k[h], 4 * st + e, scale);
#pragma unroll
            for (int n = 0; n < N; n++)
              sc[n][h] =
                  __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), qf[n][st], sc[n][h], 0, 0, 0);
          }
        fetch_k();
        const bool whole = t0 + kTile <= s.context && (t0 >= lo_most || t0 + kTile <= seen_first) && on0 && on1;
        unsigned seen[N];
        if (!whole) {
          unsigned any = 0;
#pragma unroll
          for (int n = 0; n < N; n++) {
            unsigned w = seen_word(s, t0, lo[n], seen_first, lds_mask[mask_at[n]], (int)p.a.words);
            w &= (on0 ? 0xFFFFu : 0u) | (on1 ? 0xFFFF0000u : 0u);
            seen[n] = live[n] ? w : 0u;
            any |= seen[n];
          }
#pragma unroll
          for (int k = 1; k < 16; k <<= 1) any |= (unsigned)__shfl_xor((int)any, k, 64);
          // a token that no row sees: its V bytes are whatever the page holds, so
          // its codes and scale are cleared
#pragma unroll
          for (int r = 0; r < 8; r++) {
            const bool kept = (any >> (16 * (r >> 2) + 4 * g + (r & 3))) & 1;
#pragma unroll
            for (int w = 0; w < (int)(sizeof(t.v[r]) / 4); w++) t.v[r][w] = kept ? t.v[r][w] : 0u;
            t.vs[r >> 2] = kept ? t.vs[r >> 2] : t.vs[r >> 2] & ~(0xFFu << (8 * (r & 3)));
          }
        }
        // softmax over the tile; y[4 h + r]: row i, token t0 + 16 h + 4 g + r
        u32x4 pt[N][kTerms];
#pragma unroll
        for (int n = 0; n < N; n++) {
          float y[8];
#pragma unroll
          for (int r = 0; r < 8; r++) y[r] = sc[n][r >> 2][r & 3];
          if (!whole) {
#pragma unroll
            for (int r = 0; r < 8; r++)
              y[r] = (seen[n] >> (16 * (r >> 2) + 4 * g + (r & 3))) & 1 ? y[r] : -INFINITY;
          }
          float top = y[0];
#pragma unroll
          for (int r = 1; r < 8; r++) top = fmaxf(top, y[r]);
          top = fmaxf(m[n], max_groups(top));
          const float ref = top > -INFINITY ? top * to_log2 : 0.0f;  // nothing seen yet: every p is 0
          if (__builtin_amdgcn_ballot_w64(top > m[n]) != 0) {
            // the old terms are relative to the rounded m * to_log2, so that is what
            // moves them: exactly 1 for a row whose maximum stays
            const float alpha = __builtin_amdgcn_exp2f(m[n] * to_log2 - ref);
            l[n] *= alpha;
#pragma unroll
            for (int k = 0; k < J; k++) acc[n][k] *= alpha;
            m[n] = top;
          }
          // P in bf16 terms: each takes the upper half of what the ones before
          // it left (truncated; the last one rounded)
#pragma unroll
          for (int r = 0; r < 8; r += 2) {
            float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(y[r], to_log2, -ref));
            float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(y[r + 1], to_log2, -ref));
            l[n] += p0 + p1;
#pragma unroll
            for (int k = 0; k < kTerms; k++) {
              if (k + 1 == kTerms) {
                pt[n][k][r >> 1] = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)p0, (__bf16)p1});
              } else {
                const unsigned w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
                pt[n][k][r >> 1] = perm(w1, w0, 0x07060302u);
                p0 -= __uint_as_float(w0 & 0xFFFF0000u);  // exact
                p1 -= __uint_as_float(w1 & 0xFFFF0000u);
              }
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
          if (!whole) {
            // A NaN (or an infinity) of a token that some rows see must not reach
            // the others as NaN times 0: it leaves the product, and a product of
            // ones counts, for each row and element, the seen tokens that had one
            u32x4 odd[2];
            unsigned found = 0;
#pragma unroll
            for (int o = 0; o < 2; o++)
#pragma unroll
              for (int r = 0; r < 4; r++) {
                unsigned one = 0;
                if ((va[o][r] & 0x7F80u) == 0x7F80u) one |= 0x3F80u, va[o][r] &= 0xFFFF0000u;
                if ((va[o][r] & 0x7F800000u) == 0x7F800000u) one |= 0x3F800000u, va[o][r] &= 0xFFFFu;
                odd[o][r] = one;
                found |= one;
              }
            if (__builtin_amdgcn_ballot_w64(found != 0) != 0) {
#pragma unroll
              for (int n = 0; n < N; n++) {
                u32x4 is;
#pragma unroll
                for (int r = 0; r < 4; r++) {
                  const unsigned at = 16 * (r >> 1) + 4 * g + 2 * (r & 1);
                  is[r] = ((seen[n] >> at) & 1 ? 0x3F80u : 0u) | ((seen[n] >> (at + 1)) & 1 ? 0x3F800000u : 0u);
                }
#pragma unroll
                for (int o = 0; o < 2; o++) {
                  const f32x4 hits = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                      __builtin_bit_cast(bf16x8, odd[o]), __builtin_bit_cast(bf16x8, is), (f32x4){0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
                  for (int r = 0; r < 4; r++)
                    acc[n][2 * j2 + o][r] = hits[r] > 0 ? __builtin_nanf("") : acc[n][2 * j2 + o][r];
                }
              }
            }
          }
#pragma unroll
          for (int n = 0; n < N; n++)
#pragma unroll
            for (int k = 0; k < kTerms; k++)
#pragma unroll
              for (int o = 0; o < 2; o++)
                acc[n][2 * j2 + o] =
                    __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, va[o]),
                                                            __builtin_bit_cast(bf16x8, pt[n][k]), acc[n][2 * j2 + o], 0, 0, 0);
        }
        fetch_v(j + 1);
      }
    }

    // join the waves that shared tiles, a set at a time (maxima in log2 units from here on)
    const bool opens = kRanges ? first == 0 : blockIdx.x % p.shares == 0, closes = last == s.n;  // of the unit
    const bool alone = kRanges ? opens && closes : p.shares == 1;
    if (opens && threadIdx.x == 0 && (kRanges ? !(p.by_block && closes) : !alone)) {
      const unsigned unit = ((unsigned)b * p.c.heads + head) * p.row_groups + rg;
      int* w = p.parts + 4 * (p.by_block ? blockIdx.x : unit);
      w[0] = kRanges ? (int)((u_first + (unsigned)s.n - 1) / per - blockIdx.x) + 1 : (int)p.shares;
      w[1] = (int)blockIdx.x, w[2] = (int)unit;
    }
#pragma unroll
    for (int n = 0; n < N; n++) {
      const float ln = sum_groups(l[n]), mn = m[n] * to_log2;
      if (g == 0) lds_m[wave][i] = mn;
      __syncthreads();
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWaves; w++) {
        const float mw = lds_m[w][i];
        mt = w >> per_shift == row_wave ? fmaxf(mt, mw) : mt;
      }
      const float f = mn > -INFINITY ? __builtin_amdgcn_exp2f(mn - mt) : 0.0f;
      if (g == 0) lds_l[wave][i] = ln * f;  // (no maximum: 0, or NaN if all its scores were)
      if (g == 0 && sub == 0) lds_top[wave][i] = mt;
#pragma unroll
      for (int j = 0; j < J; j++)
#pragma unroll
        for (int r = 0; r < 4; r++) lds_o[wave][i][(4 * g + r) * J + j] = acc[n][j][r] * f;
      __syncthreads();

      // out: threads over (row of the set, 4 elements)
      constexpr int kQuads = D / 4;
      for (unsigned e = threadIdx.x; e < ((unsigned)kSet << p.row_shift) * kQuads; e += kThreads) {
        const unsigned rr = e / kQuads, d4 = e % kQuads, wb = rr / kSet << per_shift;
        const unsigned in_unit = (rr / kSet * N + n) * kSet + rr % kSet, r = row0 + in_unit;
        if (r >= p.rows) continue;
        const float mx = lds_top[wb][rr % kSet];
        float sum = 0;
        f32x4 o = {0, 0, 0, 0};
#pragma unroll
        for (unsigned w = 0; w < kWaves; w++) {
          if (w >= per_tile) break;
          sum += lds_l[wb + w][rr % kSet];
          o += *(const f32x4*)&lds_o[wb + w][rr % kSet][4 * d4];
        }
        if (alone) {
          const unsigned token = r / p.group;
          const int64_t hq = (int64_t)head * p.group + (r - token * p.group);
          store_out(p.a, ((b * drafts + token) * p.a.q_heads + hq) * D + 4 * d4, finish(p.a, hq, mx, sum, o));
        } else {
          // a block has at most one part of a unit that a block before it
          // opened (slot 0) and one of a unit that it opens itself (slot 1)
          const int64_t slot = (2 * (int64_t)blockIdx.x + (opens ? 1 : 0)) * unit_rows + in_unit;
          *(f32x4*)(p.part_o + slot * D + 4 * d4) = o;
          if (d4 == 0) {
            p.part_ml[2 * slot] = mx;
            p.part_ml[2 * slot + 1] = sum;
          }
        }
      }
      if (n + 1 < N) __syncthreads();
    }
    // the next unit: the next row group, cache head or sequence
    if constexpr (!kRanges) break;
    x = u_first + (unsigned)last;
    if (x >= end) break;
    u_first = x;
    if (++rg == p.row_groups) {
      rg = 0;
      if (++head == p.c.heads) {
        head = 0;
        s = tree_span<kTile>(p, ++b);
      }
    }
    x = uniform(x), u_first = uniform(u_first), head = uniform(head), rg = uniform(rg), b = uniform((int)b);
    __syncthreads();  // it writes the same LDS
  }
}

// Many rows (65 and more of a cache head): the kW waves of a block take 32 rows
// each, of one tile of kW * 1024 / D tokens that they decode together, into LDS, as
// bf16: K by token, V by element.  (Decoded by each wave, as above, a tile costs
// more instructions than its products take.)  The 32x32x16 product S^T = K Q^T
// leaves 16 of 32 tokens of one row in a lane, which are the B operand of O^T +=
// V^T P^T for V's tokens in the order 0-3, 8-11, 4-7, 12-15 of each 16.
//
// A turn decodes the next tile, whose loads were issued a turn before, and then
// multiplies (322 us for the size above; after the products 341, loaded two tiles
// ahead 345; by half of the waves before and half after no better).  A wave's
// products wait for its exponentials; forming one set's while the next one's
// products run needs more registers than there are and spills (340 to 370).
// Scalars that stay in scalar registers matter most: page addresses in vector
// registers made a loop of each load (376).
//
// A row's reference moves only where its maximum has risen by more than 2^8 above
// it: the old terms are seldom scaled, and probabilities of up to 2^8 lose nothing.
template <int D, int kW>
struct Wide {
  static constexpr int kT = kW * 1024 / D;   // tokens of a tile: each thread decodes 16 elements of K and of V
  static constexpr int kKRow = 2 * D + 16;   // bytes of a token in LDS; the odd number of 16 spreads rows over the banks
  static constexpr int kVRow = 2 * kT;       // bytes of an element's row
  // 16-byte unit c of element d's row is at c ^ swizzle(d & 31): the 16 lanes that
  // read neighbouring elements, and those that write every fourth, use all banks
  static __device__ __forceinline__ int swizzle(int d) {
    return kT == 128 ? ((d >> 1) & 14) ^ (d & 1) ^ ((d & 2) << 2) : kT == 64 ? ((d >> 1) ^ (d >> 3)) & 7 : (d >> 2) & 3;
  }
};
struct WideFlags {
  unsigned off;     // runs of 16 tokens that are not there
  unsigned odd[4];  // tokens with a NaN or an infinity in V
};

template <int D, bool kFp4, int kTerms, int kW>
__global__ __launch_bounds__(64 * kW, 2) void k_tree_wide(TreeParams p) {
  typedef Wide<D, kW> W;
  constexpr int kT = W::kT, kRow = kFp4 ? D / 2 : D;
  constexpr int kSets = kT / 32;  // 32-token sets of a tile
  constexpr int kUnit = 32 * kW;  // rows
  constexpr int kOut = D / 32;    // 32-element sets of the output
  __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][kT * W::kKRow], lds_v[2][D * W::kVRow];
  __shared__ unsigned lds_mask[kUnit][kMaskRow], lds_any[kMaskRow];
  __shared__ int lds_depth[256], lds_far[2];
  __shared__ WideFlags flags[4];
  __shared__ unsigned lds_sum[kW];
  __shared__ int lds_at[3];

  const int lane = threadIdx.x & 63, i = lane & 31, g = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  unsigned x, end, u_first, head, rg, per = 0;
  int64_t b;
  TreeSpan span;
  if (!p.split) {
    unsigned id = blockIdx.x;
    const unsigned share = uniform(id % p.shares);
    id /= p.shares;
    rg = uniform(id % p.row_groups);
    id /= p.row_groups;
    head = uniform(id % p.c.heads);
    b = uniform(id / p.c.heads);
    span = tree_span<kT>(p, b);
    u_first = 0;
    x = (unsigned)((uint64_t)span.n * share / p.shares);
    end = (unsigned)((uint64_t)span.n * (share + 1) / p.shares);
  } else {
    const RangeStart r = range_start<kT>(p, 1, lds_sum, lds_at);
    if (r.x >= r.end) return;
    x = uniform(r.x), end = uniform(r.end), u_first = uniform(r.u_first), head = uniform(r.head), rg = uniform(r.rg), per = uniform(r.per), b = r.b;
    span = tree_span<kT>(p, b);
  }

  // What this thread decodes: of K, elements 16 kb .. of token kt; of V, elements
  // 4 vd .. of tokens vt .. vt + 3.  A wave's tokens, from wt on, are in one run of
  // 16 and so in one page: addresses are scalars and constant lane offsets.
  const int kt = threadIdx.x / (D / 16), kb = threadIdx.x % (D / 16);
  const int vt = 4 * (threadIdx.x / (D / 4)), vd = threadIdx.x % (D / 4);
  const int wt = wave * (kT / kW);
  const unsigned shift = p.c.page_shift, pmask = (1u << shift) - 1;
  const int k_off = (kt - wt) * kRow + kb * (kFp4 ? 8 : 16), ks_off = (kt - wt) * (D / 32) + kb / 2;
  const int v_off = (vt - wt) * kRow + vd * (kFp4 ? 2 : 4), vs_off = ((vd / 8) << shift) + vt - wt;

  while (true) {
    // (the loop's variables are in vector registers, where divisions leave them)
    x = uniform(x), u_first = uniform(u_first), head = uniform(head), rg = uniform(rg), b = uniform((int)b);
    const TreeSpan s = {uniform(span.context), uniform(span.end), uniform(span.a), uniform(span.b), uniform(span.n)};
    const int first = uniform(x - u_first), last = uniform(min(s.n, (int)(end - u_first)));
    const unsigned row0 = rg * kUnit, token0 = row0 / p.group;
    const unsigned drafts = (unsigned)p.a.drafts;
    if (threadIdx.x < 4) flags[threadIdx.x] = {};
    if (threadIdx.x < 2) lds_far[threadIdx.x] = threadIdx.x ? 0x7FFFFFFF : 0;
    load_masks(p, b, s, token0, (min(row0 + kUnit, p.rows) - 1) / p.group - token0 + 1, lds_mask, lds_any, lds_depth, lds_far);

    // the row of this lane
    const unsigned r = row0 + wave * 32 + i;
    const bool live = r < p.rows;
    const unsigned token = live ? r / p.group : token0, qh = head * p.group + (live ? r - token * p.group : 0);
    const float to_log2 = fmaxf(fabsf(p.a.scale) * kLog2e, 0x1p-100f);
    const unsigned q_sign = p.a.scale < 0 ? 0x80008000u : 0u;
    bf16x8 qf[D / 16];
#pragma unroll
    for (int st = 0; st < D / 16; st++) {
      u32x4 w = {0, 0, 0, 0};
      if (live) w = *(const u32x4*)(p.a.q + (b * drafts + token) * p.a.q_stride + (int64_t)qh * D + 16 * st + 8 * g);
      qf[st] = __builtin_bit_cast(bf16x8, w ^ q_sign);
    }
    // context tokens inside the windows of all rows, and of some row
    int lo_most = 0, lo_least = 0, seen_first = 0;
    if (p.a.window > 0) {
      lo_most = uniform(window_start(p, s.context, lds_far[0]));
      lo_least = uniform(window_start(p, s.context, lds_far[1]));
      seen_first = (int)min(p.a.first, (int64_t)s.context);
    }

    auto token_of = [&](int k) { return (k < s.a ? k : k - s.a + s.b) * kT; };
    // all rows see the whole tile (where its pages are there)
    auto whole = [&](int t0) { return t0 + kT <= s.context && (t0 >= lo_most || t0 + kT <= seen_first); };
    // what this lane's row sees of 32 tokens
    auto my_word = [&](int t0) {
      const int lo = p.a.window > 0 ? window_start(p, s.context, lds_depth[token]) : 0;
      return live ? seen_word(s, t0, lo, seen_first, lds_mask[token - token0], (int)p.a.words) : 0u;
    };
    const __attribute__((address_space(4))) int32_t* ids =
        (const __attribute__((address_space(4))) int32_t*)(p.a.table + b * p.a.table_stride);
    // the page of this wave's tokens in the tile to load next
    int id = -1;
    auto fetch_id = [&](int k) { id = uniform(ids[(unsigned)min(token_of(min(k, last - 1)) + wt, s.end - 1) >> shift]); };
    // a tile's codes, as loaded (zeros where there is no page)
    u32x4 raw_k;
    unsigned raw_v[4], raw_ks, raw_vs;
    int on = 0;
    auto fetch = [&](int k) {
      const int t = token_of(k) + wt;
      on = uniform(k < last && t < s.end && id >= 0 && id < p.c.pages ? 1 : 0);
      const int64_t page = (int64_t)(on ? id : 0) * p.c.heads + head, row = (page << shift) + (t & pmask);
      const __amdgpu_buffer_rsrc_t rk = panel_rsrc(p.a.kq + row * kRow, on ? 16 * kRow : 0);
      if constexpr (kFp4) {
        const u32x2 w = __builtin_amdgcn_raw_buffer_load_b64(rk, k_off, 0, 0);
        raw_k.x = w.x, raw_k.y = w.y;
      } else {
        raw_k = __builtin_amdgcn_raw_buffer_load_b128(rk, k_off, 0, 0);
      }
      raw_ks = __builtin_amdgcn_raw_buffer_load_b8(panel_rsrc(p.a.ks + row * (D / 32), on ? 16 * (D / 32) : 0), ks_off, 0, 0);
      const __amdgpu_buffer_rsrc_t rv = panel_rsrc(p.a.vq + row * kRow, on ? 16 * kRow : 0);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if constexpr (kFp4) raw_v[e] = __builtin_amdgcn_raw_buffer_load_b16(rv, v_off + e * kRow, 0, 0);
        else raw_v[e] = __builtin_amdgcn_raw_buffer_load_b32(rv, v_off + e * kRow, 0, 0);
      }
      const __amdgpu_buffer_rsrc_t rs =
          panel_rsrc(p.a.vs + page * (D / 32 << shift) + (t & pmask), on ? ((D / 32 - 1) << shift) + 16 : 0);
      raw_vs = __builtin_amdgcn_raw_buffer_load_b32(rs, vs_off, 0, 0);
    };
    // the loaded tile k, decoded: K and the values' bf16, and (after what may come
    // between) V
    unsigned dv[4][2];
    auto decode = [&](int k) {
      uint8_t* kl = lds_k[(k - first) & 1] + kt * W::kKRow + kb * 32;
      const float scale = e8m0_as_scale(raw_ks);
#pragma unroll
      for (int q = 0; q < 2; q++) {
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const unsigned w[1] = {kFp4 ? raw_k[q] : raw_k[2 * q + e / 2]};
          o[e] = decode2<kFp4>(w, kFp4 ? e : e & 1, scale);
        }
        *(u32x4*)(kl + q * 16) = o;
      }
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float vscale = e8m0_as_scale((raw_vs >> (8 * e)) & 0xFFu);
        dv[e][0] = decode2<kFp4>(&raw_v[e], 0, vscale);
        dv[e][1] = decode2<kFp4>(&raw_v[e], 1, vscale);
      }
    };
    auto store_v = [&](int k) {
      const int t0 = token_of(k);
      if (!whole(t0) || !on) {
        WideFlags& fl = flags[(k - first) & 3];
        // (a run's first tokens say it: what lies past the sequence's end is masked anyway)
        if (!on && wt % 16 == 0 && lane == 0) atomicOr(&fl.off, 1u << (wt / 16));
        // A token that no row sees: its V bytes are whatever the page holds, so it
        // counts as 0.  A NaN (or an infinity) of a token that some rows see must
        // not reach the others as NaN times 0: it is set to 0, and noted.
        const unsigned any =
            on ? seen_word(s, t0 + (vt & ~31), lo_least, seen_first, lds_any, (int)p.a.words) >> (vt & 31) : 0;
        unsigned odd = 0;
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
          for (int h = 0; h < 2; h++) {
            unsigned w = (any >> e) & 1 ? dv[e][h] : 0;
            if ((w & 0x7F80u) == 0x7F80u) odd |= 1u << e, w &= 0xFFFF0000u;
            if ((w & 0x7F800000u) == 0x7F800000u) odd |= 1u << e, w &= 0xFFFFu;
            dv[e][h] = w;
          }
        if (odd) atomicOr(&fl.odd[vt / 32], odd << (vt & 31));
      }
      uint8_t* vl = lds_v[(k - first) & 1];
      const int c = 2 * (vt / 16) + ((vt / 4) & 1), half = (vt / 8) & 1;
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int o = 0; o < 2; o++) {
          const unsigned sel = o ? 0x07060302u : 0x05040100u;
          const u32x2 w = {perm(dv[1][h], dv[0][h], sel), perm(dv[3][h], dv[2][h], sel)};
          const int el = 4 * vd + 2 * h + o;
          *(u32x2*)(vl + el * W::kVRow + (c ^ W::swizzle(el & 31)) * 16 + 8 * half) = w;
        }
    };

    float ref = -INFINITY, l = 0;  // in log2 units, and of this lane's tokens
    f32x16 acc[kOut], sc;
    u32x4 pt[2][kTerms];
#pragma unroll
    for (int o = 0; o < kOut; o++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[o][e] = 0;

    // S^T of set n of the tile in kl; element e: token 32 n + 8 (e / 4) + 4 g + e % 4
    auto scores = [&](const uint8_t* kl, int n) {
      const uint8_t* at = kl + (n * 32 + i) * W::kKRow + 16 * g;
      f32x16 o;
#pragma unroll
      for (int e = 0; e < 16; e++) o[e] = 0;
#pragma unroll
      for (int st = 0; st < D / 16; st++)
        o = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*(const bf16x8*)(at + 32 * st), qf[st], o, 0, 0, 0);
      return o;
    };
    // the masks of set n of tile k, which not all rows see whole
    auto mask_scores = [&](int k, int n, unsigned off) {
      const unsigned o2 = off >> (2 * n);
      const unsigned seen = my_word(token_of(k) + 32 * n) & ((o2 & 1 ? 0 : 0xFFFFu) | (o2 & 2 ? 0 : 0xFFFF0000u));
#pragma unroll
      for (int e = 0; e < 16; e++) sc[e] = (seen >> (8 * (e / 4) + 4 * g + e % 4)) & 1 ? sc[e] : -INFINITY;
    };
    // O^T += V^T P^T of half h of set n of the tile in vl
    auto values = [&](const uint8_t* vl, int n, int h) {
#pragma unroll
      for (int o = 0; o < kOut; o++) {
        const int c = 4 * n + 2 * h;
        const bf16x8 v = *(const bf16x8*)(vl + ((i * W::kVRow + (g ^ W::swizzle(i)) * 16) ^ (16 * c)) + 32 * o * W::kVRow);
#pragma unroll
        for (int t = 0; t < kTerms; t++)
          acc[o] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, __builtin_bit_cast(bf16x8, pt[h][t]), acc[o], 0, 0, 0);
      }
    };
    // The probabilities of the set in sc.  Returns what moves the old terms.
    auto weights = [&]() {
      float top = sc[0];
#pragma unroll
      for (int e = 1; e < 16; e++) top = fmaxf(top, sc[e]);
      const float high = max_halves(top) * to_log2;
      const bool rises = high > ref + 8;
      // (the old terms are moved by the difference of the two references: exactly)
      const float moved = rises ? high : ref, alpha = rises ? __builtin_amdgcn_exp2f(ref - high) : 1.0f;
      const float base = moved > -INFINITY ? moved : 0.0f;  // nothing seen yet: every p is 0
      ref = moved;
      l *= alpha;
      // P in bf16 terms: each takes the upper half of what the ones before it left
      // (truncated; the last one rounded)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[e], to_log2, -base));
        float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[e + 1], to_log2, -base));
        l += p0 + p1;
#pragma unroll
        for (int t = 0; t < kTerms; t++) {
          if (t + 1 == kTerms) {
            pt[e / 8][t][(e / 2) & 3] = __builtin_bit_cast(unsigned, (bf16x2){(__bf16)p0, (__bf16)p1});
          } else {
            const unsigned w0 = __float_as_uint(p0), w1 = __float_as_uint(p1);
            pt[e / 8][t][(e / 2) & 3] = perm(w1, w0, 0x07060302u);
            p0 -= __uint_as_float(w0 & 0xFFFF0000u);  // exact
            p1 -= __uint_as_float(w1 & 0xFFFF0000u);
          }
        }
      }
      return alpha;
    };
    // V elements of tile k that are no numbers, for the rows that see them
    auto odd_values = [&](int k) {
      const int t0 = token_of(k);
      if (whole(t0)) return;
#pragma unroll 1
      for (int n = 0; n < kSets; n++) {
        unsigned odd = uniform((int)flags[(k - first) & 3].odd[n]);
        const unsigned seen = odd ? my_word(t0 + 32 * n) : 0;
        while (odd) {
          const int bit = __builtin_ctz(odd), t = t0 + 32 * n + bit;
          odd &= odd - 1;
          const int64_t page = (int64_t)ids[(unsigned)t >> shift] * p.c.heads + head, row = (page << shift) + (t & pmask);
          const bool mine = (seen >> bit) & 1;
#pragma unroll
          for (int o = 0; o < kOut; o++) {
            const float scale = e8m0_as_scale(p.a.vs[((page * (D / 32) + o) << shift) + (t & pmask)]);
#pragma unroll
            for (int q = 0; q < 4; q++) {
              const int el = 32 * o + 8 * q + 4 * g;
              const uint8_t* src = p.a.vq + row * kRow + (kFp4 ? el / 2 : el);
              const unsigned w[1] = {kFp4 ? *(const uint16_t*)src : *(const unsigned*)src};
              const unsigned d0 = decode2<kFp4>(w, 0, scale), d1 = decode2<kFp4>(w, 1, scale);
              const float nan = __builtin_nanf("");
              if (mine && (d0 & 0x7F80u) == 0x7F80u) acc[o][4 * q] = nan;
              if (mine && (d0 & 0x7F800000u) == 0x7F800000u) acc[o][4 * q + 1] = nan;
              if (mine && (d1 & 0x7F80u) == 0x7F80u) acc[o][4 * q + 2] = nan;
              if (mine && (d1 & 0x7F800000u) == 0x7F800000u) acc[o][4 * q + 3] = nan;
            }
          }
        }
      }
    };

    // Tile k's K and V are at k & 1, its flags at k & 3.  It is loaded two turns and
    // decoded one turn before its own, ahead of that one's products.
    if (first < last) {  // (a share of a short sequence can be empty)
      fetch_id(first);
      fetch(first);
      fetch_id(first + 1);
      decode(first);
      store_v(first);
      fetch(first + 1);
      fetch_id(first + 2);
      __syncthreads();
    }
    const int sets = row0 + wave * 32 < p.rows ? kSets : 0;  // (a wave without rows decodes only)
    for (int k = first; k < last; k++) {
      const uint8_t *kl = lds_k[(k - first) & 1], *vl = lds_v[(k - first) & 1];
      if (k + 1 < last) {
        decode(k + 1);
        store_v(k + 1);
      }
      fetch(k + 2);
      fetch_id(k + 3);
      const unsigned off = uniform((int)flags[(k - first) & 3].off);
      const bool masked = !whole(token_of(k)) || off != 0;
#pragma unroll 1
      for (int n = 0; n < sets; n++) {
        sc = scores(kl, n);
        if (masked) mask_scores(k, n, off);
        const float alpha = weights();
        if (__builtin_amdgcn_ballot_w64(alpha != 1.0f) != 0) {
          asm volatile("");  // a branch: the products without it would be in every turn
#pragma unroll
          for (int o = 0; o < kOut; o++) acc[o] *= alpha;
        }
        values(vl, n, 0);
        values(vl, n, 1);
      }
      odd_values(k);
      if (threadIdx.x == 0) flags[(k - first + 2) & 3] = {};
      __syncthreads();
    }

    const bool opens = p.split ? first == 0 : blockIdx.x % p.shares == 0, closes = last == s.n;  // of the unit
    const bool alone = p.split ? opens && closes : p.shares == 1;
    if (opens && threadIdx.x == 0 && (p.split ? !(p.by_block && closes) : !alone)) {
      const unsigned unit = ((unsigned)b * p.c.heads + head) * p.row_groups + rg;
      int* w = p.parts + 4 * (p.by_block ? blockIdx.x : unit);
      w[0] = p.split ? (int)((u_first + (unsigned)s.n - 1) / per - blockIdx.x) + 1 : (int)p.shares;
      w[1] = (int)blockIdx.x, w[2] = (int)unit;
    }
    const float sum = sum_halves(l);
    if (live) {
      const int64_t hq = qh;
      // a block has at most one part of a unit that a block before it opened (slot
      // 0) and one of a unit that it opens itself (slot 1)
      const int64_t slot = (2 * (int64_t)blockIdx.x + (opens ? 1 : 0)) * kUnit + wave * 32 + i;
#pragma unroll
      for (int o = 0; o < kOut; o++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int el = 32 * o + 8 * q + 4 * g;
          const f32x4 v = {acc[o][4 * q], acc[o][4 * q + 1], acc[o][4 * q + 2], acc[o][4 * q + 3]};
          if (alone)
            store_out(p.a, ((b * drafts + token) * p.a.q_heads + hq) * D + el, finish(p.a, hq, ref, sum, v));
          else
            *(f32x4*)(p.part_o + slot * D + el) = v;
        }
      if (!alone && g == 0) {
        p.part_ml[2 * slot] = ref;
        p.part_ml[2 * slot + 1] = sum;
      }
    }
    // the next unit: the next row group, cache head or sequence
    if (!p.split) break;
    x = u_first + (unsigned)last;
    if (x >= end) break;
    u_first = x;
    if (++rg == p.row_groups) {
      rg = 0;
      if (++head == p.c.heads) {
        head = 0;
        span = tree_span<kT>(p, ++b);
      }
    }
    __syncthreads();  // it writes the same LDS
  }
}

// Adds the parts of the unit of record blockIdx.x, kRowsEach rows a block (grid
// y), each by kLines lines of D / 4 threads: a line adds every kLines-th part in
// order, then the lines are added in order.
template <int D, int kRowsEach>
__global__ __launch_bounds__(256) void k_tree_join(TreeParams p, unsigned unit_rows) {
  constexpr int kQuads = D / 4, kLines = 256 / kQuads / kRowsEach;
  __shared__ f32x4 lo[256 / kQuads][kQuads];
  __shared__ float ll[256 / kQuads], lm[256 / kQuads];
  const int* w = p.parts + 4 * blockIdx.x;
  const int parts = w[0];
  if (parts < 2) return;
  const unsigned k0 = w[1], unit = w[2];
  const unsigned head = unit / p.row_groups % p.c.heads;
  const int64_t b = unit / (p.row_groups * p.c.heads);
  const int d4 = threadIdx.x % kQuads, at = threadIdx.x / kQuads, line = at % kLines;
  const unsigned in_unit = blockIdx.y * kRowsEach + at / kLines, r = unit % p.row_groups * unit_rows + in_unit;
  const bool live = in_unit < unit_rows && r < p.rows;
  auto slot = [&](int part) { return (int64_t)(2 * (k0 + part) + (part == 0 ? 1 : 0)) * unit_rows + in_unit; };
  float top = -INFINITY, sum = 0;
  f32x4 o = {0, 0, 0, 0};
  if (live) {
    // a line's parts four at a time, all loads first
    constexpr int kN = 4;
    for (int k = line; k < parts; k += kN * kLines) {
      f32x2 ml[kN];
      f32x4 po[kN];
#pragma unroll
      for (int c = 0; c < kN; c++) {
        const int64_t sl = slot(min(k + c * kLines, parts - 1));
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
        if (k + c * kLines >= parts) continue;
        const float f = __builtin_amdgcn_exp2f(ml[c].x - ref);
        sum += f * ml[c].y;
        o += po[c] * f;
      }
    }
  }
  if constexpr (kLines > 1) {
    lo[at][d4] = o;
    if (d4 == 0) ll[at] = sum, lm[at] = top;
    __syncthreads();
    if (line != 0) return;
#pragma unroll
    for (int k = 1; k < kLines; k++) top = fmaxf(top, lm[at + k]);
    const float ref = top > -INFINITY ? top : 0.0f;
    o = (f32x4){0, 0, 0, 0};
    sum = 0;
#pragma unroll
    for (int k = 0; k < kLines; k++) {
      const float f = __builtin_amdgcn_exp2f(lm[at + k] - ref);
      o += lo[at + k][d4] * f;
      sum += ll[at + k] * f;
    }
  }
  if (!live) return;
  const unsigned token = r / p.group;
  const int64_t hq = (int64_t)head * p.group + (r - token * p.group);
  store_out(p.a, ((b * p.a.drafts + token) * p.a.q_heads + hq) * D + 4 * d4, finish(p.a, hq, top, sum, o));
}

}  // namespace

// Shape of a call's units.  Up to 64 rows of a cache head, k_tree_attend: N sets
// of 16 rows a wave, of one or two row waves.  More, k_tree_wide, whose blocks
// decode for 128 or 256 rows.  Measured, D = 128 E4M3, 8 cache heads: 64 rows (64
// sequences of 4600 tokens) 212 us and 328 us by k_tree_wide; 128 rows (32 of
// 4600) 215 us by k_tree_attend and 182; 512 rows (4 of 20500) 512 and 322.
struct TreeUnits {
  bool wide;
  int sets, tile, blocks;  // blocks: that take ranges, one or two a CU
  unsigned row_shift, rows, row_groups;  // rows of a unit; units per sequence and cache head
};
static TreeUnits tree_units(int64_t drafts, unsigned q_heads, const KvShape& c) {
  const int64_t rows = (int64_t)(q_heads / c.heads) * drafts;
  TreeUnits u;
  u.wide = rows > 64;
  u.sets = rows > kSet && c.dim <= 128 ? 2 : 1;
  u.row_shift = !u.wide && rows > u.sets * kSet ? 1 : 0;
  u.rows = u.wide ? (rows > 128 || c.dim == 256 ? 256 : 128) : (u.sets * kSet) << u.row_shift;
  u.row_groups = (unsigned)((rows + u.rows - 1) / u.rows);
  u.tile = u.wide ? 32 * (int)u.rows / (int)c.dim : kTile;
  u.blocks = u.wide && u.rows == 256 ? 256 : 512;
  return u;
}

// Tiles of the longest sequence that the table can name.
static int64_t tree_tiles(const TreeUnits& u, int64_t drafts, const KvShape& c, int64_t table_width, int64_t window,
                          int64_t first) {
  const int64_t most = std::min<int64_t>(table_width << c.page_shift, kMaxLen);
  int64_t tiles = (most + u.tile - 1) / u.tile;
  if (window > 0 && window < most && first < most)
    tiles = std::min(tiles, (first + u.tile - 1) / u.tile + (window + drafts) / u.tile + 2);
  return tiles;
}

// How a call's tiles are cut.  By ranges, blocks take equal runs of all units'
// tiles, whatever the sequences' lengths; a block that ends one unit and begins
// the next pays for the masks, the rows and the results of both.  By shares, a
// unit is cut in equal shares, a block each.
//
// Shares are for short calls and for one sequence, from 8 tiles a wave on: the
// second launch and the parts cost 5 us, a wave's tile of two row sets 1.1 us.  So
// cut, 8 tokens over 1000 (8 cache heads of 8 query heads, D = 128) take 20 us
// instead of 35 (27 by ranges), over 8 sequences 25 (37); by two blocks a CU these 8 take 32.
// Below 8 tiles (256 tokens, one sequence) a call takes 20 us either way.
struct TreePlan {
  bool ranges;
  unsigned shares;
  int64_t blocks;
};
static TreePlan tree_plan(const TreeUnits& u, const KvShape& c, int64_t batch, int64_t tiles) {
  const int64_t units = batch * c.heads * u.row_groups, waves = u.wide ? 1 : kWaves >> u.row_shift, each = (tiles + waves - 1) / waves;
  const bool deep = tiles * u.tile > (units >= 128 ? 2048 : 1024);
  TreePlan t = {deep && !(batch == 1 && 4 * units <= u.blocks), 1, units};
  if (t.ranges) {
    t.blocks = std::min<int64_t>(u.blocks, units * each);
  } else if (each >= 8) {
    t.shares = (unsigned)std::max<int64_t>(1, std::min((deep ? u.blocks : u.wide ? 128 : 256) / units, each / 2));
    t.blocks = units * t.shares;
  }
  return t;
}

// Blocks of a call, -1 where its tiles are too many.
int64_t tree_attend_blocks(int64_t batch, int64_t drafts, unsigned q_heads, const KvShape& c, int64_t table_width,
                           int64_t window, int64_t first) {
  const TreeUnits u = tree_units(drafts, q_heads, c);
  const int64_t tiles = tree_tiles(u, drafts, c, table_width, window, first);
  // flattened tile indexes are 32 bits, with room for one range more
  if (batch * c.heads * u.row_groups > (0x7FFFFFFF - 4096) / tiles) return -1;
  return tree_plan(u, c, batch, tiles).blocks;
}

int64_t tree_attend_workspace(int64_t batch, int64_t drafts, unsigned q_heads, const KvShape& c, int64_t table_width,
                              int64_t window, int64_t first) {
  const TreeUnits u = tree_units(drafts, q_heads, c);
  const TreePlan t = tree_plan(u, c, batch, tree_tiles(u, drafts, c, table_width, window, first));
  return t.ranges || t.shares > 1 ? t.blocks * (16 + 2 * (int64_t)u.rows * (c.dim + 2) * 4) : 0;
}

template <int D>
static void launch_join(const TreeParams& p, unsigned unit_rows, int64_t records, bool few, hipStream_t st) {
  constexpr int kLines = 256 / (D / 4), kFew = kLines > 8 ? kLines / 8 : 1;
  const unsigned rows = std::min(p.rows, unit_rows);
  if (few)
    k_tree_join<D, kLines><<<dim3((unsigned)records, (rows + kLines - 1) / kLines), dim3(256), 0, st>>>(p, unit_rows);
  else
    k_tree_join<D, kFew><<<dim3((unsigned)records, (rows + kFew - 1) / kFew), dim3(256), 0, st>>>(p, unit_rows);
}

hipError_t launch_tree_attend(const TreeArgs& a, const KvShape& c, bool fp4, void* workspace, hipStream_t st) {
  const TreeUnits u = tree_units(a.drafts, a.q_heads, c);
  TreeParams p;
  p.a = a;
  p.c = c;
  p.group = a.q_heads / c.heads;
  p.rows = p.group * (unsigned)a.drafts;
  p.row_groups = u.row_groups;
  p.row_shift = u.row_shift;
  const TreePlan t = tree_plan(u, c, a.batch, tree_tiles(u, a.drafts, c, a.table_width, a.window, a.first));
  const int64_t units = a.batch * c.heads * u.row_groups, blocks = t.blocks;
  const bool ranges = t.ranges;
  p.split = ranges;
  p.shares = t.shares;
  p.by_block = ranges && units >= blocks / 2;
  p.parts = (int*)workspace;  // at most a record a block, in either case
  p.part_o = (float*)((uint8_t*)workspace + blocks * 16);
  p.part_ml = p.part_o + 2 * blocks * u.rows * c.dim;
  const dim3 grid((unsigned)blocks), block(kThreads);
#define MXQ_TREE_R(D, F, T, N) \
  ranges ? k_tree_attend<D, F, T, N, true><<<grid, block, 0, st>>>(p) : k_tree_attend<D, F, T, N, false><<<grid, block, 0, st>>>(p)
#define MXQ_TREE_W(D, F, T, N) k_tree_wide<D, F, T, N><<<grid, dim3(64 * N), 0, st>>>(p)
#define MXQ_TREE_N(K, D, N)                          \
  do {                                               \
    if (a.bf16_out && fp4) K(D, true, 2, N);         \
    else if (a.bf16_out) K(D, false, 2, N);          \
    else if (fp4) K(D, true, 3, N);                  \
    else K(D, false, 3, N);                          \
  } while (0)
  if (u.wide) {
    if (c.dim == 64 && u.rows == 128) MXQ_TREE_N(MXQ_TREE_W, 64, 4);
    else if (c.dim == 64) MXQ_TREE_N(MXQ_TREE_W, 64, 8);
    else if (c.dim == 128 && u.rows == 128) MXQ_TREE_N(MXQ_TREE_W, 128, 4);
    else if (c.dim == 128) MXQ_TREE_N(MXQ_TREE_W, 128, 8);
    else MXQ_TREE_N(MXQ_TREE_W, 256, 8);
  } else if (c.dim == 64 && u.sets == 1) {
    MXQ_TREE_N(MXQ_TREE_R, 64, 1);
  } else if (c.dim == 64) {
    MXQ_TREE_N(MXQ_TREE_R, 64, 2);
  } else if (c.dim == 128 && u.sets == 1) {
    MXQ_TREE_N(MXQ_TREE_R, 128, 1);
  } else if (c.dim == 128) {
    MXQ_TREE_N(MXQ_TREE_R, 128, 2);
  } else {
    MXQ_TREE_N(MXQ_TREE_R, 256, 1);
  }
  if (ranges || t.shares > 1) {
    const int64_t records = p.by_block ? blocks : units;
    const bool few = blocks < 8 * units;  // parts of a unit
    if (c.dim == 64) launch_join<64>(p, u.rows, records, few, st);
    else if (c.dim == 128) launch_join<128>(p, u.rows, records, few, st);
    else launch_join<256>(p, u.rows, records, few, st);
  }
#undef MXQ_TREE_N
#undef MXQ_TREE_W
#undef MXQ_TREE_R
  return hipGetLastError();
}

}  // namespace mxq
