// sample.hip -- draw of a token from each row of logits, with temperature, top-k,
// top-p and min-p, from given random numbers (gfx950).
//
//   w_i = exp((x_i - max x) / temperature), ordered by x, equal ones by index;
//   kept: the shortest prefix of that order of those that top-k, top-p and min-p allow;
//   the token: the first by index whose running sum of kept w passes u * (their sum)
//
// Arithmetic.  Weights are fp64 and summed as whole multiples of 2^-43 of the
// largest (64-bit integers), so a sum has no order: every way of splitting it
// gives the same thresholds and the same token.  Weights below 2^-44 of the
// largest count as 0 (all of them in a row of 2^20 are below 2^-24 of it).  Order
// is that of the logits' bits as whole numbers.
#include "mxq_device.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kEach = 8;                  // elements a lane takes at a time
constexpr int kSegment = 64 * kEach;      // elements a wave takes at a time
constexpr int kMostSegments = (1 << 20) / kSegment + 1;

// One row, as groups of 8 elements on 32 (bf16: 16) byte boundaries, the first
// `lead` elements of which lie before the row.
template <bool kBf16>
struct Row {
  const uint8_t* at;  // of the first group
  int lead, vocab;
  __device__ Row(const void* logits, int64_t offset, int n) : vocab(n) {
    constexpr unsigned kSize = kBf16 ? 2 : 4;
    const uint8_t* p = (const uint8_t*)logits + offset * kSize;
    lead = (int)(((uintptr_t)p / kSize) % kEach);
    at = p - lead * kSize;
  }
  __device__ int groups() const { return (vocab + lead + kEach - 1) / kEach; }
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
};

// fp32 values in the order of their keys.
__device__ __forceinline__ unsigned key_of(float x) {
  const unsigned u = __float_as_uint(x);
  return u ^ (u >> 31 ? ~0u : 0x80000000u);
}
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k); }

// The weights of a row.
struct Weights {
  double top, inv_t;
  // exp((x - top) / t): 2^n times the Taylor polynomial of the rest, |r| <= ln 2 / 2.
  __device__ double of(float x) const {
    const double z = fmax(((double)x - top) * inv_t, -64.0);  // (also what is not a number: -inf * 0)
    const double n = __builtin_rint(z * 0x1.71547652b82fep+0);
    const double r = __builtin_fma(-n, 0x1.abc9e3b39803fp-56, __builtin_fma(-n, 0x1.62e42fefa39efp-1, z));
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, r, 1.0 / 479001600.0);
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
  }
  // w in units of 2^-43 (the last bit of numbers in [512, 1024)).
  static __device__ u64 units(double w) { return (u64)__double_as_longlong(w + 512.0) - 0x4080000000000000ull; }
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int n) { return __shfl_up(v, n, 64); }
__device__ __forceinline__ u64 sum_wave64(u64 v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// What a row keeps: keys above `key`, and the first `ties` by index of those
// that are equal to it (key 0: all); of them weights of at least min_w.
struct Kept {
  unsigned key;
  u64 ties;
  double min_w;
};

struct Shared {
  u64 mass[kMostSegments];
  unsigned ties[kMostSegments];
  u64 bin_mass[256];
  unsigned bin_count[256];
  u64 wave_sum[kWaves];
  unsigned wave_key[kWaves];
  u64 found_mass, total;
  unsigned found_count, found;
};

// The key at which the row's elements, from the largest down, reach a count (at
// least `count` of them) or a mass (double(sum) >= mass): eight bits at a time.
// Returns it with the count and mass of the keys above it.
struct Cut {
  unsigned key, count;
  u64 mass;
};
template <bool kBf16, bool kCount>
__device__ Cut cut_at(const Row<kBf16>& row, const Weights& wt, unsigned count, double mass, Shared& sh) {
  Cut c = {0, 0, 0};
  unsigned fixed = 0;  // bits of the key that are known
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) sh.bin_mass[i] = 0, sh.bin_count[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < row.groups(); i += kThreads) {
      float x[kEach];
      row.load(i, x);
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const unsigned k = key_of(x[j]);
        if ((k & fixed) != c.key) continue;
        atomicAdd(&sh.bin_count[(k >> shift) & 255], 1u);
        const u64 w = Weights::units(wt.of(x[j]));
        if (w) atomicAdd(&sh.bin_mass[(k >> shift) & 255], w);
      }
    }
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
        const u64 om = shfl_up64(bm, s);
        if (lane >= s) bn += on, bm += om;
      }
      bn += c.count - in, bm += c.mass - im;  // of what lies above this lane's bins
      int at = -1;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (at >= 0) break;
        const bool here = kCount ? bn + n[b] >= count : bn + n[b] > 0 && (double)(bm + m[b]) >= mass;
        if (here) at = b;
        else bn += n[b], bm += m[b];
      }
      const u64 who = __builtin_amdgcn_ballot_w64(at >= 0);
      if (who && lane == __builtin_ctzll(who)) sh.found = 255 - 4 * lane - at, sh.found_count = bn, sh.found_mass = bm;
    }
    __syncthreads();
    c.key |= sh.found << shift, c.count = sh.found_count, c.mass = sh.found_mass;
    fixed |= 255u << shift;
  }
  return c;
}

struct SampleParams {
  SampleArgs a;
};

// One row a block.
template <bool kBf16>
__global__ __launch_bounds__(kThreads) void k_sample(SampleParams p) {
  __shared__ Shared sh;
  const SampleArgs& a = p.a;
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Row<kBf16> row(a.logits, r * a.stride, (int)a.vocab);
  const int groups = row.groups(), segments = (groups + 63) / 64;

  // the largest, as a key (a NaN has one above all others, whatever its sign)
  unsigned top = 0;
  for (int i = threadIdx.x; i < groups; i += kThreads) {
    float x[kEach];
    row.load(i, x);
#pragma unroll
    for (int j = 0; j < kEach; j++) top = max(top, x[j] != x[j] ? ~0u : key_of(x[j]));
  }
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) top = max(top, (unsigned)__shfl_xor((int)top, m, 64));
  if (lane == 0) sh.wave_key[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; w++) top = max(top, sh.wave_key[w]);
  if (top >= key_of(INFINITY) || top <= key_of(-INFINITY)) {  // no distribution
    if (threadIdx.x == 0) a.tokens[r] = -1, a.shares[r] = __builtin_nanf("");
    return;
  }

  float t = a.temperature_of ? a.temperature_of[r] : a.temperature;
  int64_t k = a.top_k_of ? a.top_k_of[r] : a.top_k;
  const float top_p = a.top_p_of ? a.top_p_of[r] : a.top_p;
  if (!(t > 0)) t = 1, k = 1;  // the largest
  const Weights wt = {(double)of_key(top), 1.0 / (double)t};
  Kept kept = {0, ~0ull, fmin((double)(a.min_p_of ? a.min_p_of[r] : a.min_p), 1.0)};

  const bool cut_k = k > 0 && k < a.vocab, cut_p = top_p < 1;
  u64 total = 0;
  if (cut_k) {
    const Cut c = cut_at<kBf16, true>(row, wt, (unsigned)k, 0, sh);
    kept.key = c.key, kept.ties = (u64)k - c.count;
    total = c.mass + kept.ties * Weights::units(wt.of(of_key(c.key)));
  } else if (cut_p) {
    for (int i = threadIdx.x; i < groups; i += kThreads) {
      float x[kEach];
      row.load(i, x);
#pragma unroll
      for (int j = 0; j < kEach; j++) total += Weights::units(wt.of(x[j]));
    }
    total = sum_wave64(total);
    if (lane == 0) sh.wave_sum[wave] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) total += sh.wave_sum[w];
  }
  if (cut_p) {
    const double reach = (double)top_p * (double)total;
    const Cut c = cut_at<kBf16, false>(row, wt, 0, reach, sh);
    const u64 w = Weights::units(wt.of(of_key(c.key)));
    u64 n = 1;  // equal ones that it takes
    if (w > 0 && reach > (double)(c.mass + w)) n = (u64)((reach - (double)c.mass) / (double)w);
    while (w > 0 && (double)(c.mass + n * w) < reach) n++;
    while (n > 1 && (double)(c.mass + (n - 1) * w) >= reach) n--;
    kept.key = c.key, kept.ties = n;
  }
  __syncthreads();

  // kept mass by segment: of keys above the cut, and the equal ones' number
  const double w_tie = wt.of(of_key(kept.key));
  const u64 tie = kept.key && !(w_tie < kept.min_w) ? Weights::units(w_tie) : 0;
  for (int s = wave; s < segments; s += kWaves) {
    u64 m = 0;
    unsigned n = 0;
    if (s * 64 + lane < groups) {
      float x[kEach];
      row.load(s * 64 + lane, x);
#pragma unroll
      for (int j = 0; j < kEach; j++) {
        const double w = wt.of(x[j]);
        const unsigned key = key_of(x[j]);
        if (key > kept.key && !(w < kept.min_w)) m += Weights::units(w);
        n += key == kept.key;
      }
    }
    m = sum_wave64(m);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor((int)n, d, 64);
    if (lane == 0) sh.mass[s] = m, sh.ties[s] = n;
  }
  __syncthreads();
  if (wave != 0) return;
  // one wave: the segment that u falls into, then the element
  u64 sum = 0;
  unsigned ties = 0;
  for (int s0 = 0; s0 < segments; s0 += 64) {  // ties before a segment, and the sum
    const int s = s0 + lane;
    unsigned n = s < segments ? sh.ties[s] : 0, incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const unsigned o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    const u64 before = ties + (incl - n), left = kept.ties > before ? kept.ties - before : 0;
    if (s < segments) {
      sh.mass[s] += min((u64)n, left) * tie;
      sh.ties[s] = (unsigned)before;
      sum += sh.mass[s];
    }
    ties += __shfl(incl, 63, 64);
  }
  sum = sum_wave64(sum);
  const double goal = fmin(fmax((double)a.u[r], 0.0), 1.0) * (double)sum;
  u64 run = 0;
  int at = -1, last = -1;  // the segment, and the last one with any mass
  u64 run_at = 0, run_last = 0;
  for (int s0 = 0; s0 < segments && at < 0; s0 += 64) {
    const int s = s0 + lane;
    const u64 m = s < segments ? sh.mass[s] : 0;
    u64 incl = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const u64 o = shfl_up64(incl, d);
      if (lane >= d) incl += o;
    }
    const u64 some = __builtin_amdgcn_ballot_w64(m > 0);
    const u64 past = __builtin_amdgcn_ballot_w64(m > 0 && (double)(run + incl) > goal);
    const u64 before = run + incl - m;
    if (some) {
      const int l = 63 - __builtin_clzll(some);
      last = s0 + l, run_last = __shfl(before, l, 64);
    }
    if (past) {
      const int l = __builtin_ctzll(past);
      at = s0 + l, run_at = __shfl(before, l, 64);
    }
    run += __shfl(incl, 63, 64);
  }
  if (at < 0) at = last, run_at = run_last;  // u = 1: the last that may be drawn
  float x[kEach];
  u64 m[kEach], mine = 0;
  unsigned n = 0;
#pragma unroll
  for (int j = 0; j < kEach; j++) x[j] = -INFINITY;
  if (at * 64 + lane < groups) row.load(at * 64 + lane, x);
#pragma unroll
  for (int j = 0; j < kEach; j++) n += key_of(x[j]) == kept.key;
  unsigned incl_n = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned o = __shfl_up(incl_n, d, 64);
    if (lane >= d) incl_n += o;
  }
  u64 before_n = sh.ties[at] + (incl_n - n);
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    const double w = wt.of(x[j]);
    const unsigned key = key_of(x[j]);
    m[j] = 0;
    if (key > kept.key && !(w < kept.min_w)) m[j] = Weights::units(w);
    if (key == kept.key && before_n++ < kept.ties) m[j] = tie;
    mine += m[j];
  }
  u64 incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(incl, d);
    if (lane >= d) incl += o;
  }
  u64 before = run_at + incl - mine;
  int pick = -1, end = -1;
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    before += m[j];
    if (m[j] > 0) end = j;
    if (pick < 0 && m[j] > 0 && (double)before > goal) pick = j;
  }
  const u64 who = __builtin_amdgcn_ballot_w64(pick >= 0), any = __builtin_amdgcn_ballot_w64(end >= 0);
  const int owner = who ? __builtin_ctzll(who) : 63 - __builtin_clzll(any);
  if (lane == owner) {
    if (!who) pick = end;
    float chosen = x[0];
#pragma unroll
    for (int j = 1; j < kEach; j++) chosen = j == pick ? x[j] : chosen;
    a.tokens[r] = (at * 64 + lane) * kEach - row.lead + pick;
    a.shares[r] = (float)(wt.of(chosen) * 0x1p43 / (double)sum);
  }
}

}  // namespace

int64_t sample_workspace(int64_t, int64_t) { return 0; }

hipError_t launch_sample(const SampleArgs& a, bool bf16, void*, hipStream_t st) {
  SampleParams p;
  p.a = a;
  if (bf16) k_sample<true><<<dim3((unsigned)a.rows), dim3(kThreads), 0, st>>>(p);
  else k_sample<false><<<dim3((unsigned)a.rows), dim3(kThreads), 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace mxq
