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
// Rows of up to 8192 logits take one block (k_sample_row), which cuts the order
// eight bits of the logits at a time.  Longer rows are split, 8192 logits a
// block, in three launches:
//   k_sample_scan: a block's largest; and, by the row's settings, the index of
//     the largest (greedy), the weights' sums of its segments of 512 (nothing
//     cut off), or a histogram of numbers and weights over 1024 bins of 1/32 of
//     the exponent (top-k, top-p), all relative to the block's own largest;
//   k_sample_plan: a row's blocks joined: rows without a cut are finished here,
//     for others the bins that a cut can lie in;
//   k_sample_cut: a second pass that sums, by segment, what is certainly kept, and
//     lists the tokens of those bins (all down to the cut, if they are at most
//     2048); the row's last block cuts the list and draws.
// A row whose cut lies in a bin with more than 2048 tokens (equal logits, mostly)
// is left to one block of k_sample_cut, which does what k_sample_row does.
// What a row gives depends on that row alone, not on the others of the call.
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
constexpr int kBins = 1024;     // the last one: weights below e^-31.9, which count as 0
constexpr float kBinsPer = 32;  // of the exponent
constexpr int kList = 2048;

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

// Weights relative to `top`, in fp64: exp(z) = 2^n times the Taylor polynomial of
// 2^y, |y| <= 1/2 (it ends below 2^-51).
struct Weights {
  double top, per;  // log2 e / temperature
  __device__ Weights(float t, float temperature) : top((double)t), per(0x1.71547652b82fep+0 / (double)temperature) {}
  __device__ double of(float x) const {
    const double z = fmax(((double)x - top) * per, -90.0);  // (also what is not a number: -inf * 0)
    const double n = __builtin_rint(z), y = z - n;
    double p = 0x1.c3bd650fc2986p-36;  // (ln 2)^12 / 12!, and so on
    p = __builtin_fma(p, y, 0x1.e8cac7351bb25p-32);
    p = __builtin_fma(p, y, 0x1.e4cf5158b8ecap-28);
    p = __builtin_fma(p, y, 0x1.b5253d395e7c4p-24);
    p = __builtin_fma(p, y, 0x1.62c0223a5c824p-20);
    p = __builtin_fma(p, y, 0x1.ffcbfc588b0c7p-17);
    p = __builtin_fma(p, y, 0x1.430912f86c787p-13);
    p = __builtin_fma(p, y, 0x1.5d87fe78a6731p-10);
    p = __builtin_fma(p, y, 0x1.3b2ab6fba4e77p-7);
    p = __builtin_fma(p, y, 0x1.c6b08d704a0c0p-5);
    p = __builtin_fma(p, y, 0x1.ebfbdff82c58fp-3);
    p = __builtin_fma(p, y, 0x1.62e42fefa39efp-1);
    p = __builtin_fma(p, y, 1.0);
    return __builtin_ldexp(p, (int)n);
  }
  // w in units of 2^-43 (the last bit of numbers in [512, 1024)).
  static __device__ u64 units(double w) { return (u64)__double_as_longlong(w + 512.0) - 0x4080000000000000ull; }
};

// Bins of exponents: `grid` is a whole number that rises with x, and a bin is how
// far it lies below that of the largest.  Below kGridMost these are exact, so bins
// counted from a block's largest and from the row's differ by a constant.  (Rows
// whose largest is 2^19 temperatures or more from 0 are past it and left to one
// block.)
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
  unsigned found_count, found;
};

// The key at which a source's elements, from the largest down, reach a count (at
// least `count` of them) or a mass (double(sum) >= mass): eight bits at a time.
// `above` of them lie above the source.  Returns it with what lies above the key.
struct Cut {
  unsigned key, count;
  u64 mass;
};
template <bool kCount, class Source, class Mass>
__device__ Cut cut_at(const Source& src, Cut above, unsigned count, double mass, int lowest, CutLds& sh, Mass mass_of) {
  Cut c = above;
  c.key = 0;
  unsigned fixed = 0;  // bits of the key that are known
#pragma unroll 1
  for (int shift = 24; shift >= lowest; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += blockDim.x) sh.bin_mass[i] = 0, sh.bin_count[i] = 0;
    if (threadIdx.x == 0) sh.found = 0, sh.found_count = c.count, sh.found_mass = c.mass;
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
      unsigned some_n = 0;
      u64 some_m = 0;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (at >= 0) continue;
        if (n[b] > 0) some = b, some_n = bn, some_m = bm;
        if (n[b] > 0 && (kCount ? bn + n[b] >= count : (double)(bm + m[b]) >= mass)) at = b;
        bn += n[b], bm += m[b];
      }
      u64 who = __builtin_amdgcn_ballot_w64(at >= 0);
      int owner = who ? __builtin_ctzll(who) : -1;
      if (!who) {
        who = __builtin_amdgcn_ballot_w64(some >= 0);
        if (who) owner = 63 - __builtin_clzll(who);
      }
      if (lane == owner) sh.found = 255 - 4 * lane - some, sh.found_count = some_n, sh.found_mass = some_m;
    }
    __syncthreads();
    c.key |= sh.found << shift, c.count = sh.found_count, c.mass = sh.found_mass;
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
  return (int)~cut_at<true>(same, {0, 0, 0}, (unsigned)min(n, (u64)0x7FFFFFFF), 0, 0, sh, [](unsigned) { return (u64)0; }).key;
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
    ties = k - c.count;
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
  // sums of runs of 64 segments a step, in order
  double sum = 0;
  for (int s0 = 0; s0 < segments; s0 += 64) {
    double v = s0 + lane < segments ? (double)mass[s0 + lane] * scale_of(s0 + lane) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(v, d, 64);
      if (lane >= d) v += o;
    }
    sum += __shfl(v, 63, 64);
  }
  const double goal = fmin(fmax((double)a.u[r], 0.0), 1.0) * sum;
  double run = 0, run_at = 0, run_last = 0;
  int at = -1, last = 0;  // the segment, and the last one with any mass
  for (int s0 = 0; s0 < segments && at < 0; s0 += 64) {
    const u64 m = s0 + lane < segments ? mass[s0 + lane] : 0;
    double v = m ? (double)m * scale_of(s0 + lane) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_up(v, d, 64);
      if (lane >= d) v += o;
    }
    double before = __shfl_up(v, 1, 64);
    before = run + (lane ? before : 0);
    const u64 some = __builtin_amdgcn_ballot_w64(m > 0);
    const u64 past = __builtin_amdgcn_ballot_w64(m > 0 && run + v > goal);
    if (some) last = s0 + 63 - __builtin_clzll(some), run_last = __shfl(before, 63 - __builtin_clzll(some), 64);
    if (past) at = s0 + __builtin_ctzll(past), run_at = __shfl(before, __builtin_ctzll(past), 64);
    run += __shfl(v, 63, 64);
  }
  if (at < 0) at = last, run_at = run_last;  // u = 1: the last that may be drawn
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
  u64 incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = __shfl_up(incl, d, 64);
    if (lane >= d) incl += o;
  }
  u64 before = incl - mine;
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
  const Kept kept = cut_both<kBf16>(row, {0, 0, 0}, set.cut_k, (unsigned)set.k, row, {0, 0, 0}, set.cut_p, set.top_p,
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

// What the kernels of long rows hand on, a row each.
struct Plan {
  int mode;  // kDone, kListed, kAlone
  unsigned top;
  int lo, hi, bin_k;           // listed: bins lo to hi, and bin_k where top-k cuts (else -1)
  unsigned above_k, ticket;    // tokens above bin_k
  unsigned listed;
  double mass_above_k, total;  // in units of the row's largest
};
enum { kDone, kListed, kAlone };

struct SampleParams {
  SampleArgs a;
  int64_t row0;           // first row of this launch
  unsigned blocks;        // of a row
  Plan* plan;             // [rows]
  unsigned *tops, *where;  // [rows][blocks]: the largest's key, and (greedy) its index
  u64* mass;              // [rows][blocks * kBlockSegments]
  u64* bin_mass;          // [rows][blocks][kBins]
  unsigned* bin_count;
  u32x2* list;            // [rows][kList]: key, index
};

__device__ __forceinline__ void no_token(const SampleArgs& a, int64_t r) {
  a.tokens[r] = -1;
  a.shares[r] = __builtin_nanf("");
}

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_row(SampleArgs a) {
  __shared__ CutLds sh;
  __shared__ u64 mass[kBlockSegments + 1];
  const int64_t r = blockIdx.x;
  const Row<kBf16> row(a, r);
  Settings set(a, r);
  unsigned top = 0;
  for (int i = threadIdx.x; i < row.groups(); i += kThreads) {
    float x[kEach];
    row.load(i, x);
#pragma unroll
    for (int j = 0; j < kEach; j++) top = max(top, top_key(x[j]));
  }
  top = max_block(top, sh.wave_max);
  if (no_weights(top)) {
    if (threadIdx.x == 0) no_token(a, r);
    return;
  }
  if (set.greedy) {
    unsigned at = 0;  // the largest of ~index
    row.each([&](unsigned key, int index) {
      if (key == top) at = max(at, ~(unsigned)index);
    });
    at = max_block(at, sh.wave_max);
    if (threadIdx.x == 0) a.tokens[r] = (int)~at, a.shares[r] = 1;
    return;
  }
  whole_row<kBf16>(a, r, row, set, of_key(top), mass, sh);
}

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_scan(SampleParams p) {
  __shared__ unsigned lds_max[kWaves];
  __shared__ u64 bin_mass[kBins];
  __shared__ unsigned bin_count[kBins];
  const unsigned rr = blockIdx.x / p.blocks, b = blockIdx.x % p.blocks;
  const int64_t r = p.row0 + rr;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Row<kBf16> row(p.a, r);
  const Settings set(p.a, r);
  const int s0 = (int)b * kBlockSegments + wave, groups = row.groups();
  float x[kTurns][kEach];
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int g = (s0 + t * kWaves) * 64 + lane;
#pragma unroll
    for (int j = 0; j < kEach; j++) x[t][j] = -INFINITY;
    if (g < groups) row.load(g, x[t]);
  }
  unsigned top = 0;
#pragma unroll
  for (int t = 0; t < kTurns; t++)
#pragma unroll
    for (int j = 0; j < kEach; j++) top = max(top, top_key(x[t][j]));
  if (set.binned())
    for (int i = threadIdx.x; i < kBins; i += kThreads) bin_mass[i] = 0, bin_count[i] = 0;
  top = max_block(top, lds_max);
  const int64_t at = (int64_t)rr * p.blocks + b;
  if (threadIdx.x == 0) p.tops[at] = top;
  if (set.greedy) {
    unsigned best = 0;  // the largest of ~index
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++)
        if (top_key(x[t][j]) == top) best = max(best, ~(unsigned)row.index_of((s0 + t * kWaves) * 64 + lane, j));
    best = max_block(best, lds_max);
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
      for (int j = 0; j < kEach; j++) m += Weights::units(wt.of(x[t][j]));
      m = sum_wave64(m);
      if (lane == 0) p.mass[at * kBlockSegments + t * kWaves + wave] = m;
    }
  } else if (set.binned()) {
    const Bins bins(set.temperature);
    const float grid_top = bins.grid(of_key(top));
#pragma unroll
    for (int t = 0; t < kTurns; t++)
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const int bin = bins.of(x[t][j], grid_top);
        if (bin >= kBins - 1 || !(x[t][j] > -INFINITY)) continue;
        atomicAdd(&bin_count[bin], 1u);
        const u64 w = Weights::units(wt.of(x[t][j]));
        if (w) atomicAdd(&bin_mass[bin], w);
      }
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      p.bin_mass[at * kBins + i] = bin_mass[i];
      p.bin_count[at * kBins + i] = bin_count[i];
    }
  }
}

// One row a block of kBins threads.
template <bool kBf16>
__global__ __launch_bounds__(kBins) void k_sample_plan(SampleParams p) {
  __shared__ unsigned lds_max[kBins / 64];
  __shared__ double scale[kMostBlocks];
  __shared__ u64 mass[kMostBlocks * kBlockSegments];
  __shared__ double sums[kBins];     // of a bin and those above it
  __shared__ unsigned counts[kBins];
  __shared__ double wave_mass[kBins / 64];
  __shared__ unsigned wave_count[kBins / 64];
  __shared__ int found[3];
  const unsigned rr = blockIdx.x;
  const int64_t r = p.row0 + rr, first = (int64_t)rr * p.blocks;
  const SampleArgs& a = p.a;
  const Row<kBf16> row(a, r);
  const Settings set(a, r);
  const int bin = threadIdx.x, lane = bin & 63, wave = bin >> 6;
  unsigned top = 0;
  for (unsigned b = threadIdx.x; b < p.blocks; b += kBins) top = max(top, p.tops[first + b]);
  top = max_block(top, lds_max);
  Plan plan = {kDone, top, 0, -1, -1, 0, 0, 0, 0, 0};
  if (no_weights(top)) {
    if (threadIdx.x == 0) no_token(a, r), p.plan[rr] = plan;
    return;
  }
  if (set.greedy) {
    unsigned at = 0;
    for (unsigned b = threadIdx.x; b < p.blocks; b += kBins)
      if (p.tops[first + b] == top) at = max(at, ~p.where[first + b]);
    at = max_block(at, lds_max);
    if (threadIdx.x == 0) a.tokens[r] = (int)~at, a.shares[r] = 1, p.plan[rr] = plan;
    return;
  }
  const Weights wt(of_key(top), set.temperature);
  if (set.plain()) {
    for (unsigned b = threadIdx.x; b < p.blocks; b += kBins) scale[b] = wt.of(of_key(p.tops[first + b]));
    for (int s = threadIdx.x; s < row.segments(); s += kBins) mass[s] = p.mass[first * kBlockSegments + s];
    if (threadIdx.x == 0) p.plan[rr] = plan;
    __syncthreads();
    if (wave == 0)
      draw<kBf16>(a, r, row, mass, {0, 0x7FFFFFFF, 0}, [&](int s) { return scale[s / kBlockSegments]; },
                  [&](int s) { return Weights(of_key(p.tops[first + s / kBlockSegments]), set.temperature); });
    return;
  }
  plan.mode = kListed;
  if (!set.binned()) {  // min-p alone: every token by its own weight
    plan.lo = kBins;
    if (threadIdx.x == 0) p.plan[rr] = plan;
    return;
  }

  // the blocks' bins, as bins of the row
  const Bins bins(set.temperature);
  const float grid_top = bins.grid(of_key(top));
  double m = 0;
  unsigned n = 0;
  for (unsigned b = 0; b < p.blocks; b++) {
    const unsigned t = p.tops[first + b];
    const int from = bin - (int)fminf(grid_top - bins.grid(of_key(t)), (float)kBins);
    if (from < 0 || bin == kBins - 1) continue;
    n += p.bin_count[(first + b) * kBins + from];
    m += (double)p.bin_mass[(first + b) * kBins + from] * wt.of(of_key(t));
  }
  const unsigned mine = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double om = __shfl_up(m, d, 64);
    const unsigned on = __shfl_up(n, d, 64);
    if (lane >= d) m += om, n += on;
  }
  if (lane == 63) wave_mass[wave] = m, wave_count[wave] = n;
  if (threadIdx.x < 3) found[threadIdx.x] = kBins;
  __syncthreads();
  for (int w = 0; w < wave; w++) m += wave_mass[w], n += wave_count[w];
  sums[bin] = m, counts[bin] = n;
  // (a cut below the bins, where weights count as 0, is none)
  if (set.cut_k && bin < kBins - 1 && (int64_t)n >= set.k) atomicMin(&found[0], bin);
  __syncthreads();
  const bool cut_k = set.cut_k && found[0] < kBins;
  const int bin_k = cut_k ? found[0] : -1;
  const double total = sums[kBins - 1];
  if (set.cut_p) {
    // the sums here are rounded: the bins that the cut can lie in, with a margin
    const double least = cut_k ? (bin_k > 0 ? sums[bin_k - 1] : 0) : total, most = cut_k ? sums[bin_k] : total;
    if (mine > 0 && m >= (double)set.top_p * least * (1 - 1e-9)) atomicMin(&found[1], bin);
    if (mine > 0 && m >= (double)set.top_p * most * (1 + 1e-9)) atomicMin(&found[2], bin);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    int lo = bin_k, hi = bin_k;
    if (set.cut_p) {
      hi = min(found[2], cut_k ? bin_k : kBins - 2);
      lo = min(found[1], hi);
    }
    plan.bin_k = bin_k;
    plan.total = total;
    if (cut_k && bin_k > 0) plan.above_k = counts[bin_k - 1], plan.mass_above_k = sums[bin_k - 1];
    if (!cut_k && !set.cut_p) {  // top-k below the bins: all that counts
      plan.lo = kBins;
    } else if (counts[max(hi, bin_k)] <= kList) {
      plan.lo = 0, plan.hi = max(hi, bin_k);
    } else {
      plan.lo = lo, plan.hi = hi;
      const unsigned listed = counts[hi] - (lo > 0 ? counts[lo - 1] : 0) + (bin_k > hi ? counts[bin_k] - counts[bin_k - 1] : 0);
      if (listed > kList) plan.mode = kAlone;
    }
    if (!(fabsf(grid_top) < kGridMost)) plan.mode = kAlone;
    p.plan[rr] = plan;
  }
}

// A list in LDS, the elements of bins `lo` to `hi`.
struct List {
  const u32x2* at;
  int n, lo, hi;
  Bins bins;
  float grid_top;
  template <class F>
  __device__ void each(F f) const {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const u32x2 e = at[i];
      const int b = bins.of(of_key(e.x), grid_top);
      if (b >= lo && b <= hi) f(e.x, (int)e.y);
    }
  }
};

template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample_cut(SampleParams p) {
  __shared__ CutLds sh;
  __shared__ u64 mass[kMostSegments];
  __shared__ u32x2 list[kList];
  __shared__ unsigned lds_n, lds_from;
  __shared__ bool lds_last;
  const unsigned rr = blockIdx.x / p.blocks, b = blockIdx.x % p.blocks;
  const Plan plan = p.plan[rr];
  if (plan.mode == kDone || (plan.mode == kAlone && b != 0)) return;
  const int64_t r = p.row0 + rr;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  if (threadIdx.x == 0) lds_n = 0;
  __syncthreads();
  u64* row_mass = p.mass + (int64_t)rr * p.blocks * kBlockSegments;
#pragma unroll
  for (int t = 0; t < kTurns; t++) {
    const int s = (int)b * kBlockSegments + t * kWaves + wave, g = s * 64 + lane;
    float x[kEach];
#pragma unroll
    for (int j = 0; j < kEach; j++) x[j] = -INFINITY;
    if (g < row.groups()) row.load(g, x);
    u64 m = 0;
#pragma unroll
    for (int j = 0; j < kEach; j++) {
      const int bin = bins.of(x[j], grid_top);
      if (bin < plan.lo) {
        const double w = wt.of(x[j]);
        if (!(w < set.min_w)) m += Weights::units(w);
      } else if ((bin <= plan.hi || bin == plan.bin_k) && x[j] > -INFINITY) {
        const unsigned at = atomicAdd(&lds_n, 1u);
        if (at < kList) list[at] = (u32x2){key_of(x[j]), (unsigned)row.index_of(g, j)};
      }
    }
    if (plan.lo > 0) {
      m = sum_wave64(m);
      if (lane == 0) row_mass[s] = m;
    }
  }
  __syncthreads();
  const unsigned n = min(lds_n, (unsigned)kList);
  if (threadIdx.x == 0) lds_from = n ? atomicAdd(&p.plan[rr].listed, n) : 0;
  __syncthreads();
  u32x2* row_list = p.list + (int64_t)rr * kList;
  for (unsigned i = threadIdx.x; i < n; i += kThreads)
    if (lds_from + i < kList) row_list[lds_from + i] = list[i];
  // the row's last block goes on
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) lds_last = atomicAdd(&p.plan[rr].ticket, 1u) == p.blocks - 1;
  __syncthreads();
  if (!lds_last) return;
  __threadfence();

  if (threadIdx.x == 0) lds_n = min(atomicAdd(&p.plan[rr].listed, 0u), (unsigned)kList);
  __syncthreads();
  const int all = (int)lds_n, segments = row.segments();
  for (int i = threadIdx.x; i < all; i += kThreads) list[i] = row_list[i];
  u64 sure = 0;
  for (int s = threadIdx.x; s < segments; s += kThreads) {
    mass[s] = plan.lo > 0 ? row_mass[s] : 0;
    sure += mass[s];
  }
  sure = sum_block(sure, sh.wave_sum);  // (and a barrier)
  Kept kept = {0, 0x7FFFFFFF, set.min_w};
  const bool cut_k = plan.bin_k >= 0;
  if (plan.lo < kBins) {
    // top-k cuts bin_k; top-p the listed bins, above which lies what is sure (that
    // min-p has left; where it has taken some, it takes all of the list as well)
    const List in_k = {list, all, plan.bin_k, plan.bin_k, bins, grid_top};
    const List in_p = {list, all, plan.lo, plan.hi, bins, grid_top};
    u64 above = 0;
    if (cut_k) {
      if (plan.lo == 0) {
        const List over = {list, all, 0, plan.bin_k - 1, bins, grid_top};
        over.each([&](unsigned key, int) { above += Weights::units(wt.of(of_key(key))); });
        above = sum_block(above, sh.wave_sum);
      } else {
        above = (u64)plan.mass_above_k;
      }
    }
    kept = cut_both<kBf16>(in_k, {0, plan.above_k, above}, cut_k, (unsigned)set.k, in_p, {0, 0, sure}, set.cut_p, set.top_p,
                           plan.total, wt, set.min_w, sh);
    __syncthreads();
    for (int i = threadIdx.x; i < all; i += kThreads) {
      const double w = wt.of(of_key(list[i].x));
      if (kept.has(list[i].x, (int)list[i].y, w)) atomicAdd(&mass[row.segment_of((int)list[i].y)], Weights::units(w));
    }
  }
  __syncthreads();
  if (wave == 0) draw<kBf16>(a, r, row, mass, kept, [](int) { return 1.0; }, [&](int) { return wt; });
}

// Blocks of a row whose groups begin up to `lead` elements before it.
unsigned row_blocks(int64_t vocab, int lead = kEach - 1) {
  constexpr int64_t kBlock = (int64_t)kBlockSegments * kSegment;
  return (unsigned)((vocab + lead + kBlock - 1) / kBlock);
}
bool one_block(int64_t vocab) { return vocab <= 8192; }

// Workspace of a long row, and the rows of a launch: 64 MiB of it, a row at least.
int64_t row_bytes(int64_t vocab) {
  const int64_t b = row_blocks(vocab);
  return (b * (8 + kBlockSegments * 8 + kBins * 12) + (int64_t)sizeof(Plan) + kList * 8 + 15) / 16 * 16;
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
  p.bin_mass = p.mass + most * p.blocks * kBlockSegments;
  p.list = (u32x2*)(p.bin_mass + most * p.blocks * kBins);
  p.plan = (Plan*)(p.list + most * kList);
  p.bin_count = (unsigned*)(p.plan + most);
  p.tops = p.bin_count + most * p.blocks * kBins;
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
      if (!plain) k_sample_cut<true><<<all, dim3(kThreads), 0, st>>>(p);
    } else {
      k_sample_scan<false><<<all, dim3(kThreads), 0, st>>>(p);
      k_sample_plan<false><<<each, dim3(kBins), 0, st>>>(p);
      if (!plain) k_sample_cut<false><<<all, dim3(kThreads), 0, st>>>(p);
    }
  }
  return hipGetLastError();
}

}  // namespace mxq
