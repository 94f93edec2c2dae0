// sample.hip -- draw of a token from each row of logits, with temperature, top-k,
// top-p and min-p, from given random numbers (gfx950).
//
//   w_i = exp((x_i - max x) / temperature), ordered by x, equal ones by index;
//   kept: the shortest prefix of that order of those that top-k, top-p and min-p allow;
//   the token: the first by index whose running sum of kept w passes u * (their sum)
//
// Arithmetic.  Weights are fp64 and summed as whole multiples of 2^-43 of the
// largest (64-bit integers), so a sum has no order and results repeat.  Weights
// below 2^-44 of the largest count as 0 (all of them in a row of 2^20 are below
// 2^-24 of it).  Order is that of the logits' bits as whole numbers.
//
// A row's settings decide what is done.  Greedy: the index of the largest.
// Nothing cut off: the weights' sums of segments of 512 tokens, then the segment
// and the token that u falls into.  Top-k and top-p: a histogram over 512 bins of
// 1/16 of the exponent names the bins that a cut lies in (a margin covers its
// rounded weights); their tokens are listed (4096 at most) and the cut is
// found in 64 finer bins of these, whose tokens are ranked, each against all others,
// with exact sums.  A cut in a bin with more tokens than
// that (equal logits, mostly) is found eight bits of the logits at a time, in
// passes over the row (whole_row).
//
// Rows of up to about 8192 logits take one block (k_sample_row).  Longer ones are
// split, 8192 logits a block, in four launches:
//   k_sample_scan: the sums or the histogram of a block, relative to its largest;
//   k_sample_plan: a row's blocks joined: rows without a cut are finished here,
//     for others the bins that a cut can lie in;
//   k_sample_cut: a second pass that sums, by segment, what is certainly kept, and
//     lists the tokens of those bins (all down to the cut, if they fit);
//   k_sample_draw: a row's list cut, and its token drawn.
// (Joined by a ticket in k_sample_cut, whose last block of a row went on with it,
// three launches were slower: each block's release to the other chiplets cost
// more than a launch.)
// What a row gives depends on that row alone, not on the others of the call (where
// its blocks begin, on its alignment: that moves the last bits of their sums).
#include <float.h>

#include "mxq_device.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

typedef unsigned long long u64;

constexpr int kEach = 8;              // elements a lane takes at a time
constexpr int kSegment = 64 * kEach;  // elements a wave takes at a time
constexpr int kMostSegments = (1 << 20) / kSegment + 1;
constexpr int kThreads = 512;         // of the kernels that read rows
constexpr int kWaves = kThreads / 64;
constexpr int kTurns = 2;                          // segments of a wave of k_sample_scan
constexpr int kBlockSegments = kWaves * kTurns;    // 8192 logits a block
constexpr int kMostBlocks = (kMostSegments + kBlockSegments - 1) / kBlockSegments;
constexpr int kBins = kThreads;  // the last one: weights below e^-31.8, which count as 0
constexpr float kBinsPer = 16;   // of the exponent
constexpr int kList = 4096;
constexpr int kRank = kThreads;  // tokens that are ranked, one a thread
constexpr int kFew = 96;         // up to which they are ranked at once
// Up to which a row's whole list is ranked by order and by index.  k_sample_draw for
// a row of 131072, and the other way through segments: 64 tokens 6.1 us and 8.5, 96
// 8.2 and 8.6, 128 9.4 and 8.6, 192 17.3 and 9.3 (past 96 this way does not pay).
constexpr int kFewListed = 192;
// A histogram's entry: the number of tokens, and their weights in units of 2^-36
// (cut off, so up to 2^20 of them are less than 2^-16 of the largest below).
constexpr int kPackBits = 50, kPackShift = 7;
constexpr double kMargin = 0x1p-15;

// One row, as groups of 8 elements on 32 (bf16: 16) byte boundaries, the first
// `lead` elements of which lie before the row.
template <bool kBf16>
struct Row {
  const uint8_t* at;  // of the first group
  int lead, vocab;
  __device__ Row(const SampleArgs& a, int64_t r) : vocab((int)a.vocab) {
    constexpr unsigned kSize = kBf16 ? 2 : 4;
    const uint8_t* p = (const uint8_t*)a.logits + r * a.stride * kSize;
    lead = (int)(((uintptr_t)p / kSize) % kEach);
    at = p - lead * kSize;
  }
  __device__ int groups() const { return (vocab + lead + kEach - 1) / kEach; }
  __device__ int segments() const { return (groups() + 63) / 64; }
  __device__ int segment_of(int index) const { return (index + lead) / kSegment; }
  __device__ int index_of(int group, int j) const { return group * kEach - lead + j; }
  // The elements of group i as fp32 (-0 as 0), -inf outside the row.
  __device__ void load(int i, float (&x)[kEach]) const {
    const int first = i * kEach - lead;
    if (first >= 0 && first + kEach <= vocab) {
      if constexpr (kBf16) {
        const u32x4 w = ((const u32x4*)at)[i];
#pragma unroll
        for (int j = 0; j < kEach; j++) x[j] = __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16) + 0.0f;
      } else {
        const f32x4 a = ((const f32x4*)at)[2 * i], b = ((const f32x4*)at)[2 * i + 1];
#pragma unroll
        for (int j = 0; j < kEach; j++) x[j] = (j < 4 ? a[j] : b[j - 4]) + 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        x[j] = -INFINITY;
        if (first + j < 0 || first + j >= vocab) continue;
        if constexpr (kBf16) x[j] = __uint_as_float((unsigned)((const uint16_t*)at)[i * kEach + j] << 16) + 0.0f;
        else x[j] = ((const float*)at)[i * kEach + j] + 0.0f;
      }
    }
  }
  // f(key, index) for all elements, shared by the block's threads.
  template <class F>
  __device__ void each(F f) const;
};

// fp32 values in the order of their keys; a NaN's is above all others.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned u = __float_as_uint(x);
  return u ^ (u >> 31 ? ~0u : 0x80000000u);
}
__device__ __forceinline__ unsigned top_key(float x) { return x != x ? ~0u : key_of(x); }
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k); }
constexpr unsigned kKeyInf = 0xFF800000u, kKeyMinusInf = 0x007FFFFFu;
__device__ __forceinline__ bool no_weights(unsigned top) { return top >= kKeyInf || top <= kKeyMinusInf; }

template <bool kBf16>
template <class F>
__device__ void Row<kBf16>::each(F f) const {
  for (int i = threadIdx.x; i < groups(); i += blockDim.x) {
    float x[kEach];
    load(i, x);
#pragma unroll
    for (int j = 0; j < kEach; j++)
      if (x[j] > -INFINITY) f(key_of(x[j]), index_of(i, j));
  }
}

struct Settings {
  float temperature, top_p;
  int64_t k;
  double min_w;
  bool greedy, cut_k, cut_p;
  __device__ Settings(const SampleArgs& a, int64_t r) {
    temperature = a.temperature_of ? a.temperature_of[r] : a.temperature;
    k = a.top_k_of ? a.top_k_of[r] : a.top_k;
    top_p = a.top_p_of ? a.top_p_of[r] : a.top_p;
    min_w = fmin((double)(a.min_p_of ? a.min_p_of[r] : a.min_p), 1.0);
    greedy = !(temperature > 0) || k == 1;
    cut_k = k > 0 && k < a.vocab;
    cut_p = top_p < 1;
  }
  __device__ bool plain() const { return !greedy && !cut_k && !cut_p && !(min_w > 0); }
  __device__ bool binned() const { return !greedy && (cut_k || cut_p); }
};

// Weights relative to `top`, in fp64: 2^z = 2^n times the Taylor polynomial of 2^y,
// |y| <= 1/2 (it ends below 2^-51).  Its coefficients, (ln 2)^k / k!, are kept in
// scalar registers: the compiler, which sees constants, would move each into a
// vector register for each of the products (12 of about 26 instructions more).
struct Weights {
  double top, per;  // log2 e / temperature
  double c[12];
  __device__ Weights(float t, float temperature)
      : top((double)t),
        per(0x1.71547652b82fep+0 / (double)temperature),
        c{0x1.62e42fefa39efp-1,  0x1.ebfbdff82c58fp-3,  0x1.c6b08d704a0c0p-5,  0x1.3b2ab6fba4e77p-7,
          0x1.5d87fe78a6731p-10, 0x1.430912f86c787p-13, 0x1.ffcbfc588b0c7p-17, 0x1.62c0223a5c824p-20,
          0x1.b5253d395e7c4p-24, 0x1.e4cf5158b8ecap-28, 0x1.e8cac7351bb25p-32, 0x1.c3bd650fc2986p-36} {
#pragma unroll
    for (int i = 0; i < 12; i++) asm("" : "+s"(c[i]));
  }
  __device__ double of(float x) const {
    const double z = fmax(((double)x - top) * per, -90.0);  // (also what is not a number: -inf * 0)
    const double t = z + 0x1.8p52, y = z - (t - 0x1.8p52);  // n, the nearest whole number, in the low bits of t
    double p = c[11];
#pragma unroll
    for (int i = 10; i >= 0; i--) p = __builtin_fma(p, y, c[i]);
    p = __builtin_fma(p, y, 1.0);
    u32x2 w = __builtin_bit_cast(u32x2, p);
    w.y += __builtin_bit_cast(u32x2, t).x << 20;  // times 2^n
    return __builtin_bit_cast(double, w);
  }
  // w in units of 2^-43 (the last bit of numbers in [512, 1024)).
  static __device__ u64 units(double w) { return (u64)__double_as_longlong(w + 512.0) - 0x4080000000000000ull; }
};

// Bins of exponents: `grid` is a whole number that rises with x, and a bin is how
// far it lies below that of the largest.  Below kGridMost these are exact, so bins
// counted from a block's largest and from the row's differ by a constant.  (Rows
// whose largest is 2^20 temperatures or more from 0 are past it and left to passes
// over the row by one block.)
constexpr float kGridMost = 0x1p24f;
struct Bins {
  float per;
  __device__ explicit Bins(float temperature) : per(fminf(kBinsPer / temperature, 1e30f)) {}
  __device__ float grid(float x) const { return fminf(fmaxf(floorf(x * per), -FLT_MAX), FLT_MAX); }
  __device__ int of(float x, float grid_top) const { return (int)fminf(grid_top - grid(x), (float)(kBins - 1)); }
};

__device__ __forceinline__ u64 sum_wave64(u64 v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}
// Largest over the block; lds holds one a wave.  (A barrier at its end.)
__device__ __forceinline__ unsigned max_block(unsigned v, unsigned* lds) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = max(v, (unsigned)__shfl_xor((int)v, m, 64));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  for (unsigned w = 0; w < blockDim.x / 64; w++) v = max(v, lds[w]);
  __syncthreads();
  return v;
}
__device__ __forceinline__ u64 sum_block(u64 v, u64* lds) {
  v = sum_wave64(v);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (unsigned w = 0; w < blockDim.x / 64; w++) v += lds[w];
  __syncthreads();
  return v;
}

// What a row keeps: keys above `key`, and those equal to it up to index `last`;
// of them weights of at least min_w.
struct Kept {
  unsigned key;
  int last;
  double min_w;
  __device__ bool has(unsigned k, int index, double w) const {
    return (k > key || (k == key && index <= last)) && !(w < min_w);
  }
};

// LDS of cutting and drawing.
struct CutLds {
  u64 bin_mass[256];
  unsigned bin_count[256];
  u64 wave_sum[16];
  unsigned wave_max[16];
  u64 found_mass;
  unsigned found_count, found_here, found;
};

// The key at which a source's elements, from the largest down, reach a count (at
// least `count` of them) or a mass (double(sum) >= mass): eight bits at a time.
// `above` of them lie above the source.  Returns it with what lies above the key
// and the number that have it (the lowest key, where all of them do not reach).
struct Cut {
  unsigned key, count;
  u64 mass;
  unsigned here;
};
template <bool kCount, class Source, class Mass>
__device__ Cut cut_at(const Source& src, Cut above, unsigned count, double mass, int lowest, CutLds& sh, Mass mass_of) {
  Cut c = above;
  c.key = 0;
  unsigned fixed = 0;  // bits of the key that are known
#pragma unroll 1
  for (int shift = 24; shift >= lowest; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.bin_mass[i] = 0, sh.bin_count[i] = 0;
    if (threadIdx.x == 0) sh.found = 0, sh.found_here = 0, sh.found_count = c.count, sh.found_mass = c.mass;
    __syncthreads();
    src.each([&](unsigned k, int index) {
      (void)index;
      if ((k & fixed) != c.key) return;
      atomicAdd(&sh.bin_count[(k >> shift) & 255], 1u);
      const u64 w = mass_of(k);
      if (w) atomicAdd(&sh.bin_mass[(k >> shift) & 255], w);
    });
    __syncthreads();
    if (threadIdx.x < 64) {  // bins from the top: lane l has 255 - 4 l and the three below
      const int lane = threadIdx.x;
      unsigned n[4], in = 0;
      u64 m[4], im = 0;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        n[b] = sh.bin_count[255 - 4 * lane - b], m[b] = sh.bin_mass[255 - 4 * lane - b];
        in += n[b], im += m[b];
      }
      unsigned bn = in;
      u64 bm = im;
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) {
        const unsigned on = __shfl_up(bn, s, 64);
        const u64 om = __shfl_up(bm, s, 64);
        if (lane >= s) bn += on, bm += om;
      }
      bn += c.count - in, bm += c.mass - im;  // of what lies above this lane's bins
      // the first bin that reaches; where rounding leaves none, the lowest that holds any
      int at = -1, some = -1;
      unsigned some_n = 0, some_here = 0;
      u64 some_m = 0;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (at >= 0) continue;
        if (n[b] > 0) some = b, some_n = bn, some_m = bm, some_here = n[b];
        if (n[b] > 0 && (kCount ? bn + n[b] >= count : (double)(bm + m[b]) >= mass)) at = b;
        bn += n[b], bm += m[b];
      }
      u64 who = __builtin_amdgcn_ballot_w64(at >= 0);
      int owner = who ? __builtin_ctzll(who) : -1;
      if (!who) {
        who = __builtin_amdgcn_ballot_w64(some >= 0);
        if (who) owner = 63 - __builtin_clzll(who);
      }
      if (lane == owner)
        sh.found = 255 - 4 * lane - some, sh.found_count = some_n, sh.found_mass = some_m, sh.found_here = some_here;
    }
    __syncthreads();
    c.key |= sh.found << shift, c.count = sh.found_count, c.mass = sh.found_mass, c.here = sh.found_here;
    fixed |= 255u << shift;
    __syncthreads();
  }
  return c;
}

// How far down the keys are cut: bf16 keys have 16 bits, then zeros (ones below 0).
template <bool kBf16>
__device__ __forceinline__ unsigned whole_key(unsigned k) {
  return kBf16 && !(k >> 31) ? k | 0xFFFFu : k;
}

// The index of the n-th of the source's elements with this key.
template <class Source>
struct Equal {
  const Source& src;
  unsigned key;
  template <class F>
  __device__ void each(F f) const {
    const unsigned want = key;
    src.each([&](unsigned k, int index) {
      if (k == want) f(~(unsigned)index, index);
    });
  }
};
template <class Source>
__device__ int last_of(const Source& src, unsigned key, u64 n, CutLds& sh) {
  const Equal<Source> same = {src, key};
  return (int)~cut_at<true>(same, {0, 0, 0, 0}, (unsigned)min(n, (u64)0x7FFFFFFF), 0, 0, sh, [](unsigned) { return (u64)0; }).key;
}

// Cuts a source: `in_k` holds the elements among which top-k cuts, `in_p` those
// among which top-p does, with what lies above each; `total` is the mass of what
// top-k leaves where it does not cut.
template <bool kBf16, class SourceK, class SourceP>
__device__ Kept cut_both(const SourceK& in_k, Cut above_k, bool cut_k, unsigned k, const SourceP& in_p, Cut above_p,
                         bool cut_p, float top_p, double total, const Weights& wt, double min_w, CutLds& sh) {
  constexpr int kLowest = kBf16 ? 16 : 0;
  const auto mass_of = [&](unsigned key) { return Weights::units(wt.of(of_key(whole_key<kBf16>(key)))); };
  Kept kept = {0, 0x7FFFFFFF, min_w};
  u64 ties = 0;
  if (cut_k) {
    const Cut c = cut_at<true>(in_k, above_k, k, 0, kLowest, sh, mass_of);
    kept.key = whole_key<kBf16>(c.key);
    ties = min(k - c.count, c.here);  // (fewer than k tokens above -inf: all of them)
    total = (double)(c.mass + ties * mass_of(kept.key));
  }
  if (cut_p) {
    const double reach = (double)top_p * total;
    const Cut c = cut_at<false>(in_p, above_p, 0, reach, kLowest, sh, mass_of);
    const u64 w = mass_of(c.key);
    u64 n = 1;  // equal ones that it takes
    if (w > 0 && reach > (double)(c.mass + w)) n = (u64)((reach - (double)c.mass) / (double)w);
    while (w > 0 && (double)(c.mass + n * w) < reach) n++;
    while (n > 1 && (double)(c.mass + (n - 1) * w) >= reach) n--;
    // (rounded sums could put it a step past top-k's)
    const unsigned key = whole_key<kBf16>(c.key);
    if (!cut_k || key > kept.key || (key == kept.key && n < ties)) kept.key = key, ties = n;
  }
  if (cut_p) kept.last = last_of(in_p, kept.key, ties, sh);
  else if (cut_k) kept.last = last_of(in_k, kept.key, ties, sh);
  return kept;
}

// Draws from the masses of a row's segments (in LDS), by one wave.  scale_of(s)
// is what a segment's units are worth, weights_of(s) its weights.
template <bool kBf16, class Scale, class Wts>
__device__ void draw(const SampleArgs& a, int64_t r, const Row<kBf16>& row, const u64* mass, const Kept& kept,
                     Scale scale_of, Wts weights_of) {
  const int lane = threadIdx.x & 63, groups = row.groups(), segments = row.segments();
  // a lane takes a run of segments: their sum, and (last) the last one with any mass
  const int each = (segments + 63) / 64, s0 = lane * each, s1 = min(s0 + each, segments);
  double own = 0;
  int last = -1;
  for (int s = s0; s < s1; s++) {
    own += (double)mass[s] * scale_of(s);
    if (mass[s]) last = s;
  }
  double incl = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  const double sum = __shfl(incl, 63, 64), goal = fmin(fmax((double)a.u[r], 0.0), 1.0) * sum;
  double run_at = __shfl_up(incl, 1, 64);  // before the run, then before the segment
  if (lane == 0) run_at = 0;
  const u64 past = __builtin_amdgcn_ballot_w64(last >= 0 && incl > goal), some = __builtin_amdgcn_ballot_w64(last >= 0);
  const int runner = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : 0;  // (u = 1: the last)
  int at = last;
  if (lane == runner) {
    double run = run_at;
    for (int s = s0; s < s1; s++) {
      const double v = (double)mass[s] * scale_of(s);
      if (mass[s]) run_at = run;
      if (mass[s] && run + v > goal) {
        at = s;
        break;
      }
      run += v;
    }
  }
  at = max(0, __shfl(at, runner, 64)), run_at = __shfl(run_at, runner, 64);
  const double left = (goal - run_at) / scale_of(at);
  const Weights wt = weights_of(at);
  const int group = at * 64 + lane;
  float x[kEach];
  u64 m[kEach], mine = 0;
#pragma unroll
  for (int j = 0; j < kEach; j++) x[j] = -INFINITY;
  if (group < groups) row.load(group, x);
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    const double w = wt.of(x[j]);
    m[j] = kept.has(key_of(x[j]), row.index_of(group, j), w) ? Weights::units(w) : 0;
    mine += m[j];
  }
  u64 through = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = __shfl_up(through, d, 64);
    if (lane >= d) through += o;
  }
  u64 before = through - mine;
  int pick = -1, end = -1;
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    before += m[j];
    if (m[j] > 0) end = j;
    if (pick < 0 && m[j] > 0 && (double)before > left) pick = j;
  }
  const u64 who = __builtin_amdgcn_ballot_w64(pick >= 0), any = __builtin_amdgcn_ballot_w64(end >= 0);
  const int owner = who ? __builtin_ctzll(who) : any ? 63 - __builtin_clzll(any) : 0;
  if (lane == owner) {
    if (!who) pick = max(end, 0);
    float chosen = x[0];
#pragma unroll
    for (int j = 1; j < kEach; j++) chosen = j == pick ? x[j] : chosen;
    a.tokens[r] = row.index_of(group, pick);
    a.shares[r] = (float)(wt.of(chosen) * 0x1p43 * scale_of(at) / sum);
  }
}

// A row by one block, from its largest on: all passes over the row itself.
template <bool kBf16>
__device__ void whole_row(const SampleArgs& a, int64_t r, const Row<kBf16>& row, const Settings& set, float top,
                          u64* mass, CutLds& sh) {
  const Weights wt(top, set.temperature);
  u64 total = 0;
  if (set.cut_p && !set.cut_k) {
    row.each([&](unsigned key, int) { total += Weights::units(wt.of(of_key(key))); });
    total = sum_block(total, sh.wave_sum);
  }
  const Kept kept = cut_both<kBf16>(row, {0, 0, 0, 0}, set.cut_k, (unsigned)set.k, row, {0, 0, 0, 0}, set.cut_p, set.top_p,
                                    (double)total, wt, set.min_w, sh);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int s = wave; s < row.segments(); s += blockDim.x / 64) {
    u64 m = 0;
    if (s * 64 + lane < row.groups()) {
      float x[kEach];
      row.load(s * 64 + lane, x);
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const double w = wt.of(x[j]);
        if (kept.has(key_of(x[j]), row.index_of(s * 64 + lane, j), w)) m += Weights::units(w);
      }
    }
    m = sum_wave64(m);
    if (lane == 0) mass[s] = m;
  }
  __syncthreads();
  if (wave == 0)
    draw<kBf16>(a, r, row, mass, kept, [](int) { return 1.0; }, [&](int) { return wt; });
}

// One block's part of a row: the groups of its segments, one a lane and turn.
template <bool kBf16>
struct Part {
  float x[kTurns][kEach];
  int first;  // segment of turn 0 (a turn's are kWaves further on)
  __device__ Part(const Row<kBf16>& row, unsigned block)
      : first((int)block * kBlockSegments + (int)(threadIdx.x >> 6)) {
    const int groups = row.groups();
#pragma unroll
    for (int t = 0; t < kTurns; t++) {
#pragma unroll
      for (int j = 0; j < kEach; j++) x[t][j] = -INFINITY;
      if (group(t) < groups) row.load(group(t), x[t]);
    }
  }
  __device__ int segment(int t) const { return first + t * kWaves; }
  __device__ int group(int t) const { return segment(t) * 64 + (int)(threadIdx.x & 63); }
  // Key of the largest, over the block.
  __device__ unsigned top(unsigned* lds) const {
    float v = x[0][0];  // (a NaN stays)
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++) v = __builtin_elementwise_maximum(v, x[t][j]);
    return max_block(top_key(v), lds);
  }
  // Index of the first that has the key `top`, as its complement (0: none).
  __device__ unsigned first_top(const Row<kBf16>& row, unsigned top, unsigned* lds) const {
    unsigned best = 0;
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++)
        if (key_of(x[t][j]) == top) best = max(best, ~(unsigned)row.index_of(group(t), j));
    return max_block(best, lds);
  }
};

__device__ __forceinline__ u64 packed(u64 units) { return (1ull << kPackBits) + (units >> kPackShift); }
__device__ __forceinline__ unsigned packed_count(u64 v) { return (unsigned)(v >> kPackBits); }
__device__ __forceinline__ double packed_mass(u64 v) { return (double)((v & ((1ull << kPackBits) - 1)) << kPackShift); }

// Where a row's cuts lie: top-k in bin_k (-1: it does not cut), top-p in one of
// the bins p_lo to p_hi; the tokens above these, and down to the last of them.
struct Cuts {
  int bin_k, p_lo, p_hi;
  unsigned above_k, above_p, through_p, through;
};
struct FindLds {
  double sums[kBins];  // of a bin and those above it
  unsigned counts[kBins];
  double wave_mass[kBins / 64];
  unsigned wave_count[kBins / 64];
  int found[3];
};
// The first bin of which `here` holds, into *found (it holds of all after it).
__device__ __forceinline__ void first_bin(bool here, int* found) {
  const u64 who = __builtin_amdgcn_ballot_w64(here);
  if (who && (int)(threadIdx.x & 63) == __builtin_ctzll(who)) atomicMin(found, (int)threadIdx.x);
}
// m, n: weights (as rounded in a histogram) and number of this thread's bin.
__device__ Cuts find_cuts(double m, unsigned n, const Settings& set, double total, FindLds& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, bin = (int)threadIdx.x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double om = __shfl_up(m, d, 64);
    const unsigned on = __shfl_up(n, d, 64);
    if (lane >= d) m += om, n += on;
  }
  if (lane == 63) sh.wave_mass[wave] = m, sh.wave_count[wave] = n;
  if (threadIdx.x < 3) sh.found[threadIdx.x] = kBins;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBins / 64; w++)
    if (w < wave) m += sh.wave_mass[w], n += sh.wave_count[w];
  sh.sums[bin] = m, sh.counts[bin] = n;
  // (a cut below the bins, where weights count as 0, is none)
  first_bin(set.cut_k && bin < kBins - 1 && (int64_t)n >= set.k, &sh.found[0]);
  __syncthreads();
  Cuts c = {-1, 0, -1, 0, 0, 0, 0};
  if (set.cut_k && sh.found[0] < kBins) c.bin_k = sh.found[0];
  if (c.bin_k > 0) c.above_k = sh.counts[c.bin_k - 1];
  if (c.bin_k >= 0) c.through = sh.counts[c.bin_k];
  if (set.cut_p) {
    const double least = c.bin_k < 0 ? total : c.bin_k > 0 ? sh.sums[c.bin_k - 1] : 0;
    const double most = c.bin_k < 0 ? total : sh.sums[c.bin_k] * (1 + kMargin);
    first_bin(n > 0 && m >= (double)set.top_p * least * (1 - kMargin), &sh.found[1]);
    first_bin(n > 0 && m >= (double)set.top_p * most * (1 + kMargin), &sh.found[2]);
    __syncthreads();
    c.p_hi = min(sh.found[2], c.bin_k < 0 ? kBins - 2 : c.bin_k);
    c.p_lo = min(sh.found[1], c.p_hi);
    if (c.p_lo > 0) c.above_p = sh.counts[c.p_lo - 1];
    c.through_p = sh.counts[c.p_hi];
    c.through = max(c.through, c.through_p);
  }
  return c;
}

// Listed tokens in LDS, those of bins `lo` to `hi`.
struct ListLds {
  u32x2 at[kList];  // key, index
  u64 units[kList];
};
struct List {
  const ListLds& list;
  int n, lo, hi;
  Bins bins;
  float grid_top;
  // g(place, key, index)
  template <class G>
  __device__ void each_place(G g) const {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const u32x2 e = list.at[i];
      const int b = bins.of(of_key(e.x), grid_top);
      if (b >= lo && b <= hi) g(i, e.x, (int)e.y);
    }
  }
  template <class F>
  __device__ void each(F f) const {
    each_place([&](int, unsigned key, int index) { f(key, index); });
  }
  __device__ u64 mass(u64* lds) const {
    u64 m = 0;
    each_place([&](int i, unsigned, int) { m += list.units[i]; });
    return sum_block(m, lds);
  }
};

struct Range {
  unsigned lo, hi;  // of keys
};
// Tokens to rank: order (key, then the complement of the index) and units.
struct RankLds {
  u64 order[kRank], units[kRank];
  u64 order_at, mass_at, order_low, mass_low;
  unsigned n, hit;
  u64 bin_mass[64], above_mass;  // narrowing
  unsigned bin_count[64], above_count;
  Range wave_range[kWaves];
};
// The source's tokens with keys in a range into LDS; their number (above kRank:
// not all of them are there).
__device__ int gather(const List& src, Range in, RankLds& sh) {
  if (threadIdx.x == 0) sh.n = 0, sh.hit = 0;
  __syncthreads();
  src.each_place([&](int i, unsigned key, int index) {
    if (key < in.lo || key > in.hi) return;
    const unsigned at = atomicAdd(&sh.n, 1u);
    if (at >= kRank) return;
    sh.order[at] = ((u64)key << 32) | ~(unsigned)index;
    sh.units[at] = src.list.units[i];
  });
  __syncthreads();
  return (int)sh.n;
}
// The range of the source's keys.
__device__ Range range_of(const List& src, RankLds& sh) {
  Range r = {~0u, 0};
  src.each([&](unsigned key, int) { r.lo = min(r.lo, key), r.hi = max(r.hi, key); });
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    r.lo = min(r.lo, (unsigned)__shfl_xor((int)r.lo, m, 64));
    r.hi = max(r.hi, (unsigned)__shfl_xor((int)r.hi, m, 64));
  }
  if ((threadIdx.x & 63) == 0) sh.wave_range[threadIdx.x >> 6] = r;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; w++) r.lo = min(r.lo, sh.wave_range[w].lo), r.hi = max(r.hi, sh.wave_range[w].hi);
  return r;
}
// 64 bins of a range of keys: the one in which a count or a mass is reached, as
// the range of its keys; count and mass, of what lies above, are moved to it.
template <bool kCount>
__device__ Range narrow(const List& src, Range in, unsigned& count, u64& mass, unsigned k, double reach, RankLds& sh) {
  const int shift = max(0, 26 - __builtin_clz((in.hi - in.lo) | 1));
  if (threadIdx.x < 64) sh.bin_mass[threadIdx.x] = 0, sh.bin_count[threadIdx.x] = 0;
  __syncthreads();
  src.each_place([&](int i, unsigned key, int) {
    if (key < in.lo || key > in.hi) return;
    const unsigned b = (in.hi - key) >> shift;
    atomicAdd(&sh.bin_count[b], 1u);
    atomicAdd(&sh.bin_mass[b], src.list.units[i]);
  });
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const unsigned n = sh.bin_count[lane];
    unsigned bn = n;
    u64 m = sh.bin_mass[lane], bm = m;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const unsigned on = __shfl_up(bn, s, 64);
      const u64 om = __shfl_up(bm, s, 64);
      if (lane >= s) bn += on, bm += om;
    }
    u64 who = __builtin_amdgcn_ballot_w64(n > 0 && (kCount ? count + bn >= k : (double)(mass + bm) >= reach));
    const u64 some = __builtin_amdgcn_ballot_w64(n > 0);
    // (where rounding leaves none, the lowest that holds any)
    const int owner = who ? __builtin_ctzll(who) : some ? 63 - __builtin_clzll(some) : 0;
    if (lane == owner) sh.hit = lane, sh.above_count = count + (bn - n), sh.above_mass = mass + (bm - m);
  }
  __syncthreads();
  count = sh.above_count, mass = sh.above_mass;
  const unsigned b = sh.hit, hi = in.hi - (b << shift), step = (1u << shift) - 1;
  __syncthreads();
  return {hi - in.lo < step ? in.lo : hi - step, hi};
}
// The last token, in order, that is taken: the one at which a count is complete,
// or the first at which the mass is.  `count` and `mass` lie above the tokens.
struct Last {
  u64 order, mass;  // mass: of it and all above it
};
template <bool kCount>
__device__ Last rank(int n, unsigned count, u64 mass, unsigned k, double reach, RankLds& sh) {
  if ((int)threadIdx.x < n) {
    const u64 order = sh.order[threadIdx.x];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < n; j++) {
      const bool over = sh.order[j] > order;
      before += over;
      mass += over ? sh.units[j] : 0;
    }
    const u64 with = mass + sh.units[threadIdx.x];
    const bool hit = kCount ? count + before + 1 == k : (double)with >= reach && !((double)mass >= reach);
    if (hit) sh.order_at = order, sh.mass_at = with, sh.hit = 1;
    if (before == n - 1) sh.order_low = order, sh.mass_low = with;
  }
  __syncthreads();
  const Last l = sh.hit ? Last{sh.order_at, sh.mass_at} : Last{sh.order_low, sh.mass_low};
  __syncthreads();
  return l;
}

// The cut of a row whose candidates are listed.  mass_k and mass_p lie above
// bin_k and p_lo; `total` is the row's.
template <bool kBf16>
__device__ Kept cut_list(const ListLds& list, int n, const Cuts& cuts, u64 mass_k, u64 mass_p, double total,
                         const Settings& set, const Weights& wt, const Bins& bins, float grid_top, RankLds& rk, CutLds& sh) {
  const List in_k = {list, n, cuts.bin_k, cuts.bin_k, bins, grid_top}, in_p = {list, n, cuts.p_lo, cuts.p_hi, bins, grid_top};
  const bool cut_k = cuts.bin_k >= 0;
  Kept kept = {0, 0x7FFFFFFF, set.min_w};
  u64 order = 0;
  bool few = true;
  const Range whole = {0, ~0u};
  if (cut_k) {
    unsigned above = cuts.above_k;
    u64 mass = mass_k;
    int c = gather(in_k, whole, rk);
    if (c > kFew) c = gather(in_k, narrow<true>(in_k, range_of(in_k, rk), above, mass, (unsigned)set.k, 0, rk), rk);
    few = c <= kRank;
    if (few) {
      const Last l = rank<true>(c, above, mass, (unsigned)set.k, 0, rk);
      order = l.order, total = (double)l.mass;
    }
  }
  if (set.cut_p && few) {
    const double reach = fmax((double)set.top_p * total, 0.5);  // (at least one token)
    unsigned above = 0;
    u64 mass = mass_p;
    int c = gather(in_p, whole, rk);
    if (c > kFew) c = gather(in_p, narrow<false>(in_p, range_of(in_p, rk), above, mass, 0, reach, rk), rk);
    few = c <= kRank;
    if (few) order = max(order, rank<false>(c, 0, mass, 0, reach, rk).order);
  }
  if (!few)
    return cut_both<kBf16>(in_k, {0, cuts.above_k, mass_k, 0}, cut_k, (unsigned)set.k, in_p, {0, 0, mass_p, 0}, set.cut_p,
                           set.top_p, total, wt, set.min_w, sh);
  kept.key = (unsigned)(order >> 32), kept.last = (int)~(unsigned)order;
  return kept;
}

__device__ __forceinline__ void no_token(const SampleArgs& a, int64_t r) {
  a.tokens[r] = -1;
  a.shares[r] = __builtin_nanf("");
}

// Rows that one block holds.  The histogram's LDS becomes the list's, so that two
// blocks fit a CU (1024 rows of 8000, top-k and top-p: 44 us; 70 with one block a CU,
// where two took 46).
struct BinLds {
  FindLds find;
  u64 bin[kBins];
};
template <bool kBf16>
__global__ __launch_bounds__(kThreads, 4) void k_sample_row(SampleArgs a) {
  __shared__ CutLds sh;
  __shared__ union {
    BinLds bins;
    ListLds list;
  } lds;
  __shared__ RankLds rk;
  __shared__ u64 mass[kBlockSegments];
  __shared__ unsigned lds_n;
  const int64_t r = blockIdx.x;
  ListLds& list = lds.list;
  u64* bin = lds.bins.bin;
  const Row<kBf16> row(a, r);
  const Settings set(a, r);
  const Part<kBf16> part(row, 0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned top = part.top(sh.wave_max);
  if (no_weights(top)) {
    if (threadIdx.x == 0) no_token(a, r);
    return;
  }
  if (set.greedy) {
    const unsigned at = part.first_top(row, top, sh.wave_max);
    if (threadIdx.x == 0) a.tokens[r] = (int)~at, a.shares[r] = 1;
    return;
  }
  const Weights wt(of_key(top), set.temperature);
  Kept kept = {0, 0x7FFFFFFF, set.min_w};
  if (set.binned()) {
    const Bins bins(set.temperature);
    const float grid_top = bins.grid(of_key(top));
    for (int i = threadIdx.x; i < kBins; i += kThreads) bin[i] = 0;
    if (threadIdx.x == 0) lds_n = 0;
    __syncthreads();
    u64 units[kTurns][kEach], sum = 0;
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const int b = bins.of(part.x[t][j], grid_top);
        units[t][j] = Weights::units(wt.of(part.x[t][j]));
        sum += units[t][j];
        if (b < kBins - 1 && part.x[t][j] > -INFINITY) atomicAdd(&bin[b], packed(units[t][j]));
      }
    sum = sum_block(sum, sh.wave_sum);
    const Cuts cuts = find_cuts(packed_mass(bin[threadIdx.x]), packed_count(bin[threadIdx.x]), set, (double)sum, lds.bins.find);
    __syncthreads();  // (the list is written over it)
    // (rounded grids say nothing of where a cut lies, or that none does)
    const bool coarse = !(fabsf(grid_top) < kGridMost);
    if (coarse || cuts.bin_k >= 0 || set.cut_p) {
      // the candidates, and what lies above them
      u64 above_k = 0, above_p = 0;
#pragma unroll
      for (int t = 0; t < kTurns; t++)
#pragma unroll
        for (int j = 0; j < kEach; j++) {
          const int b = bins.of(part.x[t][j], grid_top);
          if (b < cuts.bin_k) above_k += units[t][j];
          if (b < cuts.p_lo) above_p += units[t][j];
          if (!(b == cuts.bin_k || (b >= cuts.p_lo && b <= cuts.p_hi)) || !(part.x[t][j] > -INFINITY)) continue;
          const unsigned at = atomicAdd(&lds_n, 1u);
          if (at >= kList) continue;
          list.at[at] = (u32x2){key_of(part.x[t][j]), (unsigned)row.index_of(part.group(t), j)};
          list.units[at] = units[t][j];
        }
      above_k = sum_block(above_k, sh.wave_sum);
      above_p = sum_block(above_p, sh.wave_sum);  // (and barriers)
      if (coarse || lds_n > kList) {
        whole_row<kBf16>(a, r, row, set, of_key(top), mass, sh);
        return;
      }
      kept = cut_list<kBf16>(list, (int)lds_n, cuts, above_k, above_p, (double)sum, set, wt, bins, grid_top, rk, sh);
    }
  }
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    u64 m = 0;
#pragma unroll
    for (int j = 0; j < kEach; j++) {
      const double w = wt.of(part.x[t][j]);
      if (kept.has(key_of(part.x[t][j]), row.index_of(part.group(t), j), w)) m += Weights::units(w);
    }
    m = sum_wave64(m);
    if (lane == 0) mass[part.segment(t)] = m;
  }
  __syncthreads();
  if (wave == 0) draw<kBf16>(a, r, row, mass, kept, [](int) { return 1.0; }, [&](int) { return wt; });
}

// What the kernels of long rows hand on, a row each.
struct Plan {
  int mode;
  unsigned top;
  int lo;              // bins above it are kept but for min-p; those from it on are listed
  int all;             // all bins down to the cuts are listed
  int need_k;          // bins above bin_k are neither sure nor listed
  unsigned listed;
  Cuts cuts;
  double total;        // the row's weights, in units of its largest
  u64 mass_k;          // (need_k) of the bins above bin_k
};
enum { kDone, kListed, kAlone };

struct SampleParams {
  SampleArgs a;
  int64_t row0;            // first row of this launch
  unsigned blocks;         // of a row
  Plan* plan;              // [rows]
  unsigned *tops, *where;  // [rows][blocks]: the largest's key, and (greedy) its index
  u64* mass;               // [rows][blocks][kBlockSegments]; with a histogram, [0] is the block's sum
  u64* bins;               // [rows][blocks][kBins]
  u32x2* list;             // [rows][kList]: key, index
};

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_scan(SampleParams p) {
  __shared__ unsigned lds_max[kWaves];
  __shared__ u64 lds_sum[kWaves];
  __shared__ u64 bin[kBins];
  const unsigned rr = blockIdx.x / p.blocks, b = blockIdx.x % p.blocks;
  const int64_t r = p.row0 + rr;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Row<kBf16> row(p.a, r);
  const Settings set(p.a, r);
  const Part<kBf16> part(row, b);
  if (set.binned())
    for (int i = threadIdx.x; i < kBins; i += kThreads) bin[i] = 0;
  const unsigned top = part.top(lds_max);
  const int64_t at = (int64_t)rr * p.blocks + b;
  if (threadIdx.x == 0) p.tops[at] = top;
  if (set.greedy) {
    const unsigned best = part.first_top(row, top, lds_max);
    if (threadIdx.x == 0) p.where[at] = ~best;
    return;
  }
  if (top >= kKeyInf) return;
  const Weights wt(of_key(top), set.temperature);
  if (set.plain()) {
#pragma unroll
    for (int t = 0; t < kTurns; t++) {
      u64 m = 0;
#pragma unroll
      for (int j = 0; j < kEach; j++) m += Weights::units(wt.of(part.x[t][j]));
      m = sum_wave64(m);
      if (lane == 0) p.mass[at * kBlockSegments + t * kWaves + wave] = m;
    }
  } else if (set.binned()) {
    const Bins bins(set.temperature);
    const float grid_top = bins.grid(of_key(top));
    u64 sum = 0;
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const int i = bins.of(part.x[t][j], grid_top);
        if (i >= kBins - 1 || !(part.x[t][j] > -INFINITY)) continue;
        const u64 units = Weights::units(wt.of(part.x[t][j]));
        sum += units;
        atomicAdd(&bin[i], packed(units));
      }
    sum = sum_block(sum, lds_sum);
    if (threadIdx.x == 0) p.mass[at * kBlockSegments] = sum;
    for (int i = threadIdx.x; i < kBins; i += kThreads) p.bins[at * kBins + i] = bin[i];
  }
}

// One row a block of kBins threads.
template <bool kBf16>
__global__ __launch_bounds__(kBins) void k_sample_plan(SampleParams p) {
  __shared__ unsigned lds_max[kBins / 64];
  __shared__ unsigned tops[kMostBlocks];
  __shared__ double scale[kMostBlocks];  // of a block's units
  __shared__ int shift[kMostBlocks];     // of its bins
  __shared__ u64 mass[kMostBlocks * kBlockSegments];
  __shared__ FindLds find;
  const unsigned rr = blockIdx.x;
  const int64_t r = p.row0 + rr, first = (int64_t)rr * p.blocks;
  const SampleArgs& a = p.a;
  const Row<kBf16> row(a, r);
  const Settings set(a, r);
  unsigned top = 0;
  for (unsigned b = threadIdx.x; b < p.blocks; b += kBins) top = max(top, tops[b] = p.tops[first + b]);
  top = max_block(top, lds_max);
  Plan plan = {kDone, top, kBins, 0, 0, 0, {-1, 0, -1, 0, 0, 0, 0}, 0, 0};
  if (no_weights(top)) {
    if (threadIdx.x == 0) no_token(a, r), p.plan[rr] = plan;
    return;
  }
  if (set.greedy) {
    unsigned at = 0;
    for (unsigned b = threadIdx.x; b < p.blocks; b += kBins)
      if (tops[b] == top) at = max(at, ~p.where[first + b]);
    at = max_block(at, lds_max);
    if (threadIdx.x == 0) a.tokens[r] = (int)~at, a.shares[r] = 1, p.plan[rr] = plan;
    return;
  }
  const Weights wt(of_key(top), set.temperature);
  const Bins bins(set.temperature);
  const float grid_top = bins.grid(of_key(top));
  for (unsigned b = threadIdx.x; b < p.blocks; b += kBins) {
    const float t = of_key(tops[b]);
    scale[b] = wt.of(t);
    shift[b] = (int)fminf(grid_top - bins.grid(t), (float)kBins);
  }
  if (set.plain()) {
    for (int s = threadIdx.x; s < row.segments(); s += kBins) mass[s] = p.mass[first * kBlockSegments + s];
    if (threadIdx.x == 0) p.plan[rr] = plan;
    __syncthreads();
    if (threadIdx.x < 64)
      draw<kBf16>(a, r, row, mass, {0, 0x7FFFFFFF, 0}, [&](int s) { return scale[s / kBlockSegments]; },
                  [&](int s) { return Weights(of_key(tops[s / kBlockSegments]), set.temperature); });
    return;
  }
  plan.mode = kListed;
  if (set.binned()) {
    __syncthreads();
    // the blocks' bins, as bins of the row
    const int mine = threadIdx.x;
    double m = 0, total = 0;
    unsigned n = 0;
#pragma unroll 8
    for (unsigned b = 0; b < p.blocks; b++) {
      const int from = mine - shift[b];
      const bool any = from >= 0 && mine < kBins - 1;
      const u64 v = p.bins[(first + b) * kBins + (any ? from : 0)];
      n += any ? packed_count(v) : 0;
      m += any ? packed_mass(v) * scale[b] : 0;
      total += (double)p.mass[(first + b) * kBlockSegments] * scale[b];
    }
    const Cuts cuts = find_cuts(m, n, set, total, find);
    plan.cuts = cuts;
    plan.total = total;
    // the bin in which weights fall below min-p, or one after it
    const int bin_m = set.min_w > 0 ? (int)fminf(1 - kBinsPer * logf((float)set.min_w), (float)kBins) + 2 : kBins;
    if ((cuts.bin_k < 0 || bin_m < cuts.bin_k) && (!set.cut_p || bin_m < cuts.p_lo)) {
      // no cut but min-p's: every token by its own weight (or top-k's lies below
      // the bins, and all that counts is kept)
    } else if (cuts.through <= kList) {
      plan.lo = 0, plan.all = 1;
    } else {
      plan.lo = set.cut_p ? cuts.p_lo : cuts.bin_k;
      unsigned listed = set.cut_p ? cuts.through_p - cuts.above_p : 0;
      if (cuts.bin_k > cuts.p_hi) listed += cuts.through - cuts.above_k;
      plan.need_k = set.cut_p && cuts.bin_k > cuts.p_hi;
      if (listed > kList) plan.mode = kAlone;
    }
    if (!(fabsf(grid_top) < kGridMost)) plan.mode = kAlone;
  }  // else min-p alone: every token by its own weight
  if (threadIdx.x == 0) p.plan[rr] = plan;
}

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_cut(SampleParams p) {
  __shared__ u64 lds_sum[kWaves];
  __shared__ u32x2 list[kList];
  __shared__ unsigned lds_n, lds_from;
  const unsigned rr = blockIdx.x / p.blocks, b = blockIdx.x % p.blocks;
  const Plan plan = p.plan[rr];
  if (plan.mode != kListed) return;
  const int64_t r = p.row0 + rr;
  const int lane = threadIdx.x & 63;
  const Row<kBf16> row(p.a, r);
  const Settings set(p.a, r);
  const Part<kBf16> part(row, b);
  const Weights wt(of_key(plan.top), set.temperature);
  const Bins bins(set.temperature);
  const float grid_top = bins.grid(of_key(plan.top));
  const Cuts& cuts = plan.cuts;
  const int list_hi = plan.all ? max(cuts.p_hi, cuts.bin_k) : cuts.p_hi;
  if (threadIdx.x == 0) lds_n = 0;
  __syncthreads();
  u64* row_mass = p.mass + (int64_t)rr * p.blocks * kBlockSegments;
  u64 above_k = 0;
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    u64 m = 0;
#pragma unroll
    for (int j = 0; j < kEach; j++) {
      const float x = part.x[t][j];
      const int i = bins.of(x, grid_top);
      if (i < plan.lo || (plan.need_k && i < cuts.bin_k)) {
        const double w = wt.of(x);
        if (i < plan.lo && !(w < set.min_w)) m += Weights::units(w);
        above_k += Weights::units(w);
      }
      if (i >= plan.lo && (i <= list_hi || i == cuts.bin_k) && x > -INFINITY) {
        const unsigned at = atomicAdd(&lds_n, 1u);
        if (at < kList) list[at] = (u32x2){key_of(x), (unsigned)row.index_of(part.group(t), j)};
      }
    }
    if (plan.lo > 0) {
      m = sum_wave64(m);
      if (lane == 0) row_mass[part.segment(t)] = m;
    }
  }
  if (plan.need_k) {
    above_k = sum_block(above_k, lds_sum);
    if (threadIdx.x == 0) atomicAdd(&p.plan[rr].mass_k, above_k);
  }
  __syncthreads();
  const unsigned n = min(lds_n, (unsigned)kList);
  if (threadIdx.x == 0) lds_from = n ? atomicAdd(&p.plan[rr].listed, n) : 0;
  __syncthreads();
  u32x2* row_list = p.list + (int64_t)rr * kList;
  for (unsigned i = threadIdx.x; i < n; i += kThreads)
    if (lds_from + i < kList) row_list[lds_from + i] = list[i];
}

// A row whose tokens down to its cuts are all listed, at most kFewListed of them: each
// is ranked against all others, once by order, for the cuts, and once by index,
// for the draw.  Several threads share a token's comparisons.
struct FewLds {
  u64 order[kThreads], units[kThreads], mass[kThreads];  // mass: of the tokens before it, in order or by index
  unsigned before[kThreads];
  u64 order_k, mass_k, order_p, sum;
};
__device__ void draw_few(const SampleArgs& a, int64_t r, const u32x2* listed, int n, const Settings& set, const Cuts& cuts,
                         double total, const Weights& wt, FewLds& sh) {
  const int t = threadIdx.x;
  int width = 64;
  while (width < n) width *= 2;
  const int c = t & (width - 1), parts = kThreads / width, part = t / width;
  if (t < n) {
    const u32x2 e = listed[t];
    sh.order[t] = ((u64)e.x << 32) | ~e.y;
    sh.units[t] = Weights::units(wt.of(of_key(e.x)));
  }
  sh.mass[t] = 0, sh.before[t] = 0;
  if (t == 0) sh.order_k = sh.order_p = sh.sum = 0;
  __syncthreads();
  const u64 order = c < n ? sh.order[c] : 0, own = c < n ? sh.units[c] : 0;
  if (c < n) {
    unsigned before = 0;
    u64 mass = 0;
#pragma unroll 4
    for (int j = part; j < n; j += parts) {
      const bool over = sh.order[j] > order;
      before += over;
      mass += over ? sh.units[j] : 0;
    }
    if (before) atomicAdd(&sh.before[c], before), atomicAdd(&sh.mass[c], mass);
  }
  __syncthreads();
  const u64 mass = sh.mass[c];
  if (t < n && cuts.bin_k >= 0 && (int64_t)sh.before[t] + 1 == set.k) sh.order_k = order, sh.mass_k = mass + own;
  __syncthreads();
  sh.mass[t] = 0;
  if (set.cut_p) {
    const double reach = fmax((double)set.top_p * (cuts.bin_k >= 0 ? (double)sh.mass_k : total), 0.5);
    if (t < n && (double)(mass + own) >= reach && !((double)mass >= reach)) sh.order_p = order;
    __syncthreads();
  }
  const bool kept = c < n && order >= max(sh.order_k, sh.order_p) && !(wt.of(of_key((unsigned)(order >> 32))) < set.min_w);
  __syncthreads();
  if (t < width) sh.units[t] = kept ? own : 0;
  if (t < n && kept) atomicAdd(&sh.sum, own);
  __syncthreads();
  if (kept) {
    u64 first = 0;
#pragma unroll 4
    for (int j = part; j < n; j += parts) first += (unsigned)sh.order[j] >= (unsigned)order ? sh.units[j] : 0;
    if (first) atomicAdd(&sh.mass[c], first);
  }
  __syncthreads();
  if (t >= n || !kept || own == 0) return;
  const u64 run = sh.mass[t], sum = sh.sum;
  const double goal = fmin(fmax((double)a.u[r], 0.0), 1.0) * (double)sum;
  // (u = 1: the last)
  if (((double)run > goal && !((double)(run - own) > goal)) || (run == sum && !((double)sum > goal))) {
    a.tokens[r] = (int)~(unsigned)order;
    a.shares[r] = (float)(wt.of(of_key((unsigned)(order >> 32))) * 0x1p43 / (double)sum);
  }
}

// The lists are cut, and the tokens drawn: one row a block.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_draw(SampleParams p) {
  __shared__ CutLds sh;
  __shared__ u64 mass[kMostSegments];
  __shared__ ListLds list;
  __shared__ RankLds rk;
  __shared__ FewLds few;
  const unsigned rr = blockIdx.x;
  const Plan plan = p.plan[rr];
  if (plan.mode == kDone) return;
  const int64_t r = p.row0 + rr;
  const SampleArgs& a = p.a;
  const Row<kBf16> row(a, r);
  const Settings set(a, r);
  if (plan.mode == kAlone) {
    whole_row<kBf16>(a, r, row, set, of_key(plan.top), mass, sh);
    return;
  }
  const Weights wt(of_key(plan.top), set.temperature);
  const Bins bins(set.temperature);
  const float grid_top = bins.grid(of_key(plan.top));
  const Cuts& cuts = plan.cuts;
  const u64* row_mass = p.mass + (int64_t)rr * p.blocks * kBlockSegments;
  const u32x2* row_list = p.list + (int64_t)rr * kList;
  const int all = (int)min(plan.listed, (unsigned)kList);
  if (plan.all && all <= kFewListed) {
    draw_few(a, r, row_list, all, set, cuts, plan.total, wt, few);
    return;
  }
  for (int i = threadIdx.x; i < all; i += kThreads) {
    list.at[i] = row_list[i];
    list.units[i] = Weights::units(wt.of(of_key(list.at[i].x)));
  }
  u64 sure = 0;
  for (int s = threadIdx.x; s < row.segments(); s += kThreads) {
    mass[s] = plan.lo > 0 ? row_mass[s] : 0;
    sure += mass[s];
  }
  sure = sum_block(sure, sh.wave_sum);  // (and barriers)
  Kept kept = {0, 0x7FFFFFFF, set.min_w};
  if (plan.lo < kBins) {
    // What lies above the cuts.  (Where min-p has taken some of the sure tokens, it
    // takes all that are listed too, and where top-p cuts them says nothing.)
    u64 mass_k = sure, mass_p = sure;
    if (plan.all) {
      mass_k = List{list, all, 0, cuts.bin_k - 1, bins, grid_top}.mass(sh.wave_sum);
      mass_p = List{list, all, 0, cuts.p_lo - 1, bins, grid_top}.mass(sh.wave_sum);
    } else if (plan.need_k) {
      mass_k = plan.mass_k;
    } else if (set.cut_p && cuts.bin_k >= 0) {  // bin_k is one of top-p's bins
      mass_k = sure + List{list, all, plan.lo, cuts.bin_k - 1, bins, grid_top}.mass(sh.wave_sum);
    }
    kept = cut_list<kBf16>(list, all, cuts, mass_k, mass_p, plan.total, set, wt, bins, grid_top, rk, sh);
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += kThreads) {
      const u32x2 e = list.at[i];
      if (kept.has(e.x, (int)e.y, wt.of(of_key(e.x)))) atomicAdd(&mass[row.segment_of((int)e.y)], list.units[i]);
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) draw<kBf16>(a, r, row, mass, kept, [](int) { return 1.0; }, [&](int) { return wt; });
}

// Blocks of a row whose groups begin up to `lead` elements before it.
unsigned row_blocks(int64_t vocab, int lead = kEach - 1) {
  constexpr int64_t kBlock = (int64_t)kBlockSegments * kSegment;
  return (unsigned)((vocab + lead + kBlock - 1) / kBlock);
}
bool one_block(int64_t vocab) { return row_blocks(vocab) == 1; }

// Workspace of a long row, and the rows of a launch: 64 MiB of it, a row at least.
int64_t row_bytes(int64_t vocab) {
  const int64_t b = row_blocks(vocab);
  return (b * (8 + kBlockSegments * 8 + kBins * 8) + (int64_t)sizeof(Plan) + kList * 8 + 15) / 16 * 16;
}
int64_t rows_at_once(int64_t rows, int64_t vocab) {
  return std::min(rows, std::max<int64_t>(1, ((int64_t)64 << 20) / row_bytes(vocab)));
}

}  // namespace

int64_t sample_workspace(int64_t rows, int64_t vocab) {
  return one_block(vocab) ? 0 : rows_at_once(rows, vocab) * row_bytes(vocab);
}

hipError_t launch_sample(const SampleArgs& a, bool bf16, void* workspace, hipStream_t st) {
  if (one_block(a.vocab)) {
    if (bf16) k_sample_row<true><<<dim3((unsigned)a.rows), dim3(kThreads), 0, st>>>(a);
    else k_sample_row<false><<<dim3((unsigned)a.rows), dim3(kThreads), 0, st>>>(a);
    return hipGetLastError();
  }
  const int64_t most = rows_at_once(a.rows, a.vocab);
  SampleParams p;
  p.a = a;
  const bool same = a.rows == 1 || a.stride % kEach == 0;  // all rows begin alike
  p.blocks = row_blocks(a.vocab, same ? (int)((uintptr_t)a.logits / (bf16 ? 2 : 4) % kEach) : kEach - 1);
  p.mass = (u64*)workspace;
  p.bins = p.mass + most * p.blocks * kBlockSegments;
  p.list = (u32x2*)(p.bins + most * p.blocks * kBins);
  p.plan = (Plan*)(p.list + most * kList);
  p.tops = (unsigned*)(p.plan + most);
  p.where = p.tops + most * p.blocks;
  // (a row without a cut is finished by the second launch)
  const bool plain = !a.temperature_of && a.temperature > 0 && !a.top_k_of && (a.top_k <= 0 || a.top_k >= a.vocab) &&
                     !a.top_p_of && a.top_p >= 1 && !a.min_p_of && !(a.min_p > 0);
  for (p.row0 = 0; p.row0 < a.rows; p.row0 += most) {
    const unsigned rows = (unsigned)std::min(most, a.rows - p.row0);
    const dim3 all(rows * p.blocks), each(rows);
    if (bf16) {
      k_sample_scan<true><<<all, dim3(kThreads), 0, st>>>(p);
      k_sample_plan<true><<<each, dim3(kBins), 0, st>>>(p);
      if (plain) continue;
      k_sample_cut<true><<<all, dim3(kThreads), 0, st>>>(p);
      k_sample_draw<true><<<each, dim3(kThreads), 0, st>>>(p);
    } else {
      k_sample_scan<false><<<all, dim3(kThreads), 0, st>>>(p);
      k_sample_plan<false><<<each, dim3(kBins), 0, st>>>(p);
      if (plain) continue;
      k_sample_cut<false><<<all, dim3(kThreads), 0, st>>>(p);
      k_sample_draw<false><<<each, dim3(kThreads), 0, st>>>(p);
    }
  }
  return hipGetLastError();
}

}  // namespace mxq
