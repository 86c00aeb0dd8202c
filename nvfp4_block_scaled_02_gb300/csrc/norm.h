// norm.h -- parameter blocks of the residual norm and its gradient (norm.cu).
#pragma once
#include "kv.h"

namespace nvfp4 {

constexpr int kNormMaxCols = 16384;

struct NormParams {
  const uint4 *x, *res;    // bf16 [R][C]; res may be null
  const uint4* w;          // bf16 [C]
  int64_t R;
  int32_t C;
  float eps;
  uint4 *h, *y;            // bf16 [R][C] or null
  const float* gamax;      // one outer scale for the tensor, or null: one for each row
  float M;
  float* row_amax;         // [R] (without gamax)
  uint8_t *codes, *scales;
  uint32_t* choice;        // [R][ceil(C / 512)] or null
  uint4* dq;               // bf16 [R][C] or null
  int32_t* status;
};
// target 0 = MXFP8, 1 = NVFP4
cudaError_t launch_norm(const NormParams& p, int target, bool fos, cudaStream_t st);

struct NormBwdParams {
  const uint4 *gy, *h, *w, *gh;  // gh may be null
  int64_t R;
  int32_t C;
  float eps;
  uint4* gx;
  float* gw;                     // [C]
  float* part;                   // [CTAs][C]
  int32_t* status;
};
constexpr int64_t kNormPart = 4 << 20;  // floats of partial weight gradients at most
constexpr size_t kNormWsBytes = (size_t)4 * kNormPart;
cudaError_t launch_norm_bwd(const NormBwdParams& p, cudaStream_t st);

}  // namespace nvfp4
