// mxq_kv.h -- device helpers of the paged cache's kernels.
#pragma once
#include "mxq_device.h"

namespace mxq {

// 8 stored values (8 E4M3 bytes, or 4 bytes of E2M1 pairs in w.x) times the
// block's scale as bf16.  Exact: E4M3 and E2M1 have at most 4 significant
// bits, and the scale is a power of two (codes whose product leaves bf16's
// exponent range are outside the library's contract).
template <bool kFp4>
__device__ __forceinline__ void kv_decode8(u32x2 w, float scale, bf16x8& o) {
  bf16x2 p0, p1, p2, p3;
  if constexpr (kFp4) {
    p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.x, scale, 0);
    p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.x, scale, 1);
    p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.x, scale, 2);
    p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w.x, scale, 3);
  } else {
    p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, false);
    p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, true);
    p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, false);
    p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, true);
  }
  o = (bf16x8){p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

}  // namespace mxq
