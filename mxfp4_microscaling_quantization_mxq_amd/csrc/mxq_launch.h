// mxq_launch.h -- host-side launchers of the library's kernels (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace mxq {

// A paged cache: `pages` pages of 2^page_shift tokens, `heads` key/value
// heads of `dim` elements.
struct KvShape {
  int64_t pages;
  unsigned heads, dim, page_shift;
};

// r = x + residual (r = x without one), y = r / sqrt(mean r^2 + eps) * weight,
// (q[rows][k], s[rows][k/32]) = MXFP8(y).
hipError_t launch_rmsnorm_quantize_fp8(const void* x, const void* residual, const void* weight, bool bf16,
                                       int64_t rows, int64_t k, float eps, void* r, uint8_t* q, uint8_t* s,
                                       hipStream_t st);
// New tokens' keys and values (row strides in elements) quantized into their
// slots, and the slots' values read back.
hipError_t launch_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride, bool bf16,
                            const int64_t* slots, int64_t tokens, const KvShape& c, bool fp4, uint8_t* kq, uint8_t* ks,
                            uint8_t* vq, uint8_t* vs, hipStream_t st);
hipError_t launch_kv_read(const uint8_t* kq, const uint8_t* ks, const uint8_t* vq, const uint8_t* vs,
                          const int64_t* slots, int64_t tokens, const KvShape& c, bool fp4, void* k, void* v,
                          bool bf16, hipStream_t st);

// Attention of one new token per sequence over the paged cache.
struct AttendArgs {
  const uint16_t* q;  // bf16 [batch][q_heads][dim], rows q_stride elements apart
  int64_t q_stride;
  const uint8_t *kq, *ks, *vq, *vs;
  const int32_t* table;  // [batch][table_width], rows table_stride apart
  int64_t table_width, table_stride;
  const int32_t* lens;  // [batch]
  const float* sinks;   // [q_heads] or null
  int64_t batch, window;
  unsigned q_heads;
  float scale;
  void* out;  // [batch][q_heads][dim]
  bool bf16_out;
};
// Blocks of such a call (-1 where its tiles of 32 tokens, over all sequences
// at the table's width and all cache heads, pass 2^31), and the bytes of
// workspace that its partial results take.
int64_t attend_blocks(int64_t batch, unsigned q_heads, const KvShape& c, bool fp4, int64_t table_width, int64_t window);
int64_t attend_workspace(int64_t batch, unsigned q_heads, const KvShape& c, int64_t table_width, int64_t window);
hipError_t launch_attend(const AttendArgs& a, const KvShape& c, bool fp4, void* workspace, hipStream_t st);

hipError_t launch_mx_quantize(const void* x, bool bf16, int64_t rows, int64_t k, uint8_t* q, uint8_t* s,
                              hipStream_t st);
// MXFP8: q[rows][k] E4M3 codes, s[rows][k/32] E8M0 codes.
hipError_t launch_mx8_quantize(const void* x, bool bf16, int64_t rows, int64_t k, uint8_t* q, uint8_t* s,
                               hipStream_t st);
// W4A8: c[m][n] = sum_k A8_hat[m][k] * B4_hat[n][k], A MXFP8 (aq8[m][k],
// as[m][k/32]), B MXFP4; fp32 accumulation; c as fp32 or bf16.
hipError_t launch_w4a8(const uint8_t* aq8, const uint8_t* as, const uint8_t* bq, const uint8_t* bs, int64_t m,
                       int64_t n, int64_t k, void* c, bool bf16_out, hipStream_t st);
// MXFP4 of x rotated block by block along k with the orthonormal Hadamard
// H_hk, hk in {16, 32, 64, 128}, k % max(32, hk) == 0.
hipError_t launch_mx_quantize_hadamard(const void* x, bool bf16, int64_t rows, int64_t k, int hk, uint8_t* q,
                                       uint8_t* s, hipStream_t st);
hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t k, void* y,
                                bool bf16, hipStream_t st);
hipError_t launch_nv_quantize(const void* x, bool bf16, int64_t rows, int64_t k, float* gscale,
                              bool compute_gscale, uint8_t* q, uint8_t* s, hipStream_t st);
hipError_t launch_tf4_quantize(const void* x, bool bf16, int64_t rows, int64_t k, float* gscale,
                               bool compute_gscale, uint8_t* q, uint8_t* s, uint8_t* meta, uint16_t* res,
                               hipStream_t st);
hipError_t launch_tf4_dequantize(const uint8_t* q, const uint8_t* s, const uint8_t* meta, const uint16_t* res,
                                 const float* gscale, int64_t rows, int64_t k, void* y, bool bf16_out,
                                 hipStream_t st);
hipError_t launch_nv_dequantize(const uint8_t* q, const uint8_t* s, const float* gscale, int64_t rows,
                                int64_t k, void* y, bool bf16, hipStream_t st);

// W4A16: y[m][n] = (gscale ? *gscale : 1) * sum_k x[m][k] * deq(W)[n][k].
// nv == false: MXFP4 weight (E8M0 per 32); nv == true: NVFP4 (E4M3 per 16).
hipError_t launch_w4a16(bool nv, const uint8_t* wq, const uint8_t* ws, const float* gscale, int64_t n,
                        int64_t k, const void* x, int64_t m, void* y, bool bf16_out, hipStream_t st);

// W4A4: c[m][n] = sum_k deq(A)[m][k] * deq(B)[n][k] on the block-scaled MFMA.
hipError_t launch_w4a4(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs, int64_t m,
                       int64_t n, int64_t k, void* c, bool bf16_out, hipStream_t st);

// W4A4 and W4A8 for few activation rows (weight-stream bound), used where
// gemm_skinny_applies: m <= 128, k % 512 == 0, k <= 2^24.
bool gemm_skinny_applies(int64_t m, int64_t k);
hipError_t launch_w4a4_skinny(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                              int64_t m, int64_t n, int64_t k, void* c, bool bf16_out, hipStream_t st);
hipError_t launch_w4a8_skinny(const uint8_t* aq8, const uint8_t* as, const uint8_t* bq, const uint8_t* bs,
                              int64_t m, int64_t n, int64_t k, void* c, bool bf16_out, hipStream_t st);
// W4A4 with bf16 activations x[m][k] quantized to MXFP4 inside the kernel:
// bit-identical to launch_mx_quantize followed by launch_w4a4.  For
// 1 <= m <= 16 where gemm_skinny_applies.
hipError_t launch_w4a4_dynamic(const uint16_t* x, const uint8_t* bq, const uint8_t* bs, int64_t m, int64_t n,
                               int64_t k, void* c, bool bf16_out, hipStream_t st);
// W4A8 with bf16 activations quantized to MXFP8 inside the kernel:
// bit-identical to launch_mx8_quantize followed by launch_w4a8.  For
// 1 <= m <= 16 where gemm_skinny_applies.
hipError_t launch_w4a8_dynamic(const uint16_t* x, const uint8_t* bq, const uint8_t* bs, int64_t m, int64_t n,
                               int64_t k, void* c, bool bf16_out, hipStream_t st);

// W4A4 with the product rounded to bf16 and quantized to MXFP4 along n in
// the epilogue: cq[m][n/2], cs[m][n/32]; n % 32 == 0.
hipError_t launch_w4a4_mx(const uint8_t* aq, const uint8_t* as, const uint8_t* bq, const uint8_t* bs, int64_t m,
                          int64_t n, int64_t k, uint8_t* cq, uint8_t* cs, hipStream_t st);

}  // namespace mxq
