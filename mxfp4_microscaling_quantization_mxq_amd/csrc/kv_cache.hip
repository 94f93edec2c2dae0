// kv_cache.hip -- write of new keys and values into a paged MXFP8 / MXFP4
// cache, and its read back (gfx950).
//
// Layout (P tokens a page, a power of two; D the head size, D % 32 == 0):
//   kq, vq [pages][heads][P][D] E4M3 codes, or [P][D/2] packed E2M1 codes
//   ks     [pages][heads][P][D/32] E8M0 codes
//   vs     [pages][heads][D/32][P] E8M0 codes
// A page's share of one head is contiguous, which is what the attention
// reads; blocks run along D, so a token is quantized when it is written and
// never again.  The value scales of a block are contiguous over tokens
// because the attention's lanes hold one 32-block and eight tokens each.
//
// A token's place is its slot, page * P + position in the page.
#include "mxq_device.h"
#include "mxq_kv.h"
#include "mxq_launch.h"

namespace mxq {

namespace {

// A block takes U chunks of 256 lanes of one head (token by token, dim / 8 lanes
// each), keys or values, and issues all their loads first: neighbouring threads
// take neighbouring tokens of ONE head, whose codes and scales are neighbours
// in the page, so whole lines are written (read).  Heads, then keys and values,
// vary fastest over the grid: blocks that run together share the tokens' rows.
struct KvBlock {
  unsigned head, i0;
  bool value;
};
template <int U>
__device__ __forceinline__ KvBlock kv_block(const KvShape& c) {
  const unsigned head = blockIdx.x % c.heads, rest = blockIdx.x / c.heads;
  return {head, (rest >> 1) * (256u * U) + threadIdx.x, (rest & 1) != 0};
}

// One lane = 8 consecutive elements of one token's head; a quad of lanes = one
// block, quantized by the functions the quantizers use, so the codes are those
// of mxq_quantize / mxq_quantize_fp8.  A quad's lanes share the token, so
// skipping a slot keeps quads whole.  Measured: 16384 tokens x 8 heads x 128
// from a fused projection of 10240 bf16 into MXFP8 pages of 64: 23.1 us (4.4
// TB/s, median of a kernel trace).  Variants in turn, in one graph's replays:
// 23.5 as it is, 26.6 with a token's heads side by side in a block, 22.5 with
// four chunks a block, 23.2 without any scale store, so the scattered
// bytes of vs cost next to nothing.
template <bool kBf16, bool kFp4>
__global__ __launch_bounds__(256) void k_kv_append(const void* __restrict__ k, int64_t k_stride,
                                                   const void* __restrict__ v, int64_t v_stride,
                                                   const int64_t* __restrict__ slots, unsigned lanes, KvShape c,
                                                   uint8_t* __restrict__ kq, uint8_t* __restrict__ ks,
                                                   uint8_t* __restrict__ vq, uint8_t* __restrict__ vs) {
  const KvBlock kb = kv_block<1>(c);
  if (kb.i0 >= lanes) return;
  const unsigned head = kb.head, per_head = c.dim / 8, token = kb.i0 / per_head, in_head = kb.i0 % per_head;
  const int64_t slot = slots[token];
  if (slot < 0 || slot >= c.pages << c.page_shift) return;
  const int64_t at = (int64_t)token * (kb.value ? v_stride : k_stride) + 8 * (head * per_head + in_head);
  unsigned code;
  u32x2 out;
  if constexpr (kBf16) {
    const bf16x8 xb = __builtin_nontemporal_load((const bf16x8*)((const uint16_t*)(kb.value ? v : k) + at));
    if constexpr (kFp4) out.x = mx_quantize_quad_bf16(xb, &code);
    else out = mx8_quantize_quad_bf16(xb, &code);
  } else {
    const f32x4* p = (const f32x4*)((const float*)(kb.value ? v : k) + at);
    const f32x4 a = p[0], b = p[1];
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (kFp4) out.x = mx_quantize_quad_f32(x, &code);
    else out = mx8_quantize_quad_f32(x, &code);
  }
  const int64_t ph = (slot >> c.page_shift) * c.heads + head;
  const int64_t pos = slot & ((1 << c.page_shift) - 1);
  const int64_t lane8 = ((ph << c.page_shift) + pos) * per_head + in_head;
  uint8_t* q = kb.value ? vq : kq;
  if constexpr (kFp4) ((unsigned*)q)[lane8] = out.x;
  else ((u32x2*)q)[lane8] = out;
  if ((in_head & 3) == 0) {
    const int64_t nb = c.dim / 32, b = in_head >> 2;
    if (kb.value) vs[((ph * nb + b) << c.page_shift) + pos] = (uint8_t)code;
    else ks[((ph << c.page_shift) + pos) * nb + b] = (uint8_t)code;
  }
}

// One lane = 8 elements of one token's head.  A slot outside the cache reads
// as zeros.  32768 tokens x 8 heads x 128 to bf16: MXFP8 31.0 us (6.5 TB/s),
// MXFP4 26.5 (medians of a kernel trace).  Variants in turn, in one graph's
// replays: 35.3 and 30.1 as it is, one chunk a block 38.5 and 34.3, plain
// output stores 49.0 and 30.7.
template <bool kBf16, bool kFp4, int U>
__global__ __launch_bounds__(256) void k_kv_read(const uint8_t* __restrict__ kq, const uint8_t* __restrict__ ks,
                                                 const uint8_t* __restrict__ vq, const uint8_t* __restrict__ vs,
                                                 const int64_t* __restrict__ slots, unsigned lanes, KvShape c,
                                                 void* __restrict__ k, void* __restrict__ v) {
  const KvBlock kb = kv_block<U>(c);
  const bool value = kb.value;
  const unsigned head = kb.head, per_head = c.dim / 8, i0 = kb.i0;
  u32x2 w[U];
  unsigned code[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const unsigned i = i0 + 256u * u;
    w[u] = (u32x2){0, 0};
    code[u] = 127;
    if (i >= lanes) continue;
    const int64_t slot = slots[i / per_head];
    if (slot < 0 || slot >= c.pages << c.page_shift) continue;
    const unsigned in_head = i % per_head;
    const int64_t ph = (slot >> c.page_shift) * c.heads + head;
    const int64_t pos = slot & ((1 << c.page_shift) - 1);
    const int64_t lane8 = ((ph << c.page_shift) + pos) * per_head + in_head;
    const uint8_t* q = value ? vq : kq;
    if constexpr (kFp4) w[u].x = ((const unsigned*)q)[lane8];
    else w[u] = ((const u32x2*)q)[lane8];
    const int64_t nb = c.dim / 32, b = in_head >> 2;
    code[u] = value ? vs[((ph * nb + b) << c.page_shift) + pos] : ks[((ph << c.page_shift) + pos) * nb + b];
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    const unsigned i = i0 + 256u * u;
    if (i >= lanes) break;
    const float scale = e8m0_as_scale(code[u]);
    void* dst = value ? v : k;
    const int64_t o8 = ((int64_t)(i / per_head) * c.heads + head) * per_head + i % per_head;
    if constexpr (kBf16) {
      bf16x8 o;
      kv_decode8<kFp4>(w[u], scale, o);
      __builtin_nontemporal_store(o, &((bf16x8*)dst)[o8]);
    } else {
      f32x4 a, b;
      if constexpr (kFp4) {
        const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u].x, scale, 0);
        const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u].x, scale, 1);
        const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u].x, scale, 2);
        const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u].x, scale, 3);
        a = (f32x4){p0[0], p0[1], p1[0], p1[1]};
        b = (f32x4){p2[0], p2[1], p3[0], p3[1]};
      } else {
        const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[u].x, scale, false);
        const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[u].x, scale, true);
        const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[u].y, scale, false);
        const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[u].y, scale, true);
        a = (f32x4){p0[0], p0[1], p1[0], p1[1]};
        b = (f32x4){p2[0], p2[1], p3[0], p3[1]};
      }
      ((f32x4*)dst)[2 * o8] = a;
      ((f32x4*)dst)[2 * o8 + 1] = b;
    }
  }
}

// Chunks a block of the read, and the lanes from which it has more than one
// (fewer would leave CUs without a block).
constexpr int kReadU = 2;
constexpr int64_t kReadMany = 1 << 19;

// Tokens per launch: below 2^31 threads.
int64_t tokens_per_launch(const KvShape& c) { return ((int64_t)1 << 30) / ((int64_t)c.heads * (c.dim / 8)); }

}  // namespace

hipError_t launch_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, bool bf16,
                            const int64_t* slots, int64_t tokens, const KvShape& c, bool fp4, uint8_t* kq, uint8_t* ks,
                            uint8_t* vq, uint8_t* vs, hipStream_t st) {
  const int64_t most = tokens_per_launch(c);
  const int e = bf16 ? 2 : 4;
  for (int64_t t = 0; t < tokens; t += most) {
    const unsigned lanes = (unsigned)(std::min(most, tokens - t) * (c.dim / 8));
    const dim3 grid((lanes + 255) / 256 * 2 * c.heads), block(256);
    const void* kt = (const uint8_t*)k + t * k_stride * e;
    const void* vt = (const uint8_t*)v + t * v_stride * e;
#define MXQ_APPEND(B, F) \
  k_kv_append<B, F><<<grid, block, 0, st>>>(kt, k_stride, vt, v_stride, slots + t, lanes, c, kq, ks, vq, vs)
    if (bf16 && fp4) MXQ_APPEND(true, true);
    else if (bf16) MXQ_APPEND(true, false);
    else if (fp4) MXQ_APPEND(false, true);
    else MXQ_APPEND(false, false);
#undef MXQ_APPEND
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const uint8_t* kq, const uint8_t* ks, const uint8_t* vq, const uint8_t* vs,
                          const int64_t* slots, int64_t tokens, const KvShape& c, bool fp4, void* k, void* v,
                          bool bf16, hipStream_t st) {
  const int64_t per_token = (int64_t)c.heads * (c.dim / 8), most = tokens_per_launch(c);
  for (int64_t t = 0; t < tokens; t += most) {
    const unsigned lanes = (unsigned)(std::min(most, tokens - t) * (c.dim / 8));
    const bool few = (int64_t)lanes * c.heads < kReadMany;
    const unsigned per_block = 256 * (few ? 1 : kReadU);
    const dim3 grid((lanes + per_block - 1) / per_block * 2 * c.heads), block(256);
    const int64_t at = t * per_token * (bf16 ? 16 : 32);
    void* kt = (uint8_t*)k + at;
    void* vt = (uint8_t*)v + at;
#define MXQ_READ(B, F)                                                                              \
  few ? k_kv_read<B, F, 1><<<grid, block, 0, st>>>(kq, ks, vq, vs, slots + t, lanes, c, kt, vt)     \
      : k_kv_read<B, F, kReadU><<<grid, block, 0, st>>>(kq, ks, vq, vs, slots + t, lanes, c, kt, vt)
    if (bf16 && fp4) MXQ_READ(true, true);
    else if (bf16) MXQ_READ(true, false);
    else if (fp4) MXQ_READ(false, true);
    else MXQ_READ(false, false);
#undef MXQ_READ
  }
  return hipGetLastError();
}

}  // namespace mxq
