// api_linear.cu -- the C ABI of the quantised linear layer's operators: argument
// validation (all synchronous, before anything is enqueued) and dispatch.
#include <cmath>
#include <cstdint>

#include "matmul.h"
#include "norm.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
nvfp4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }
constexpr int64_t kMaxI32 = INT32_MAX;

// Sizes of a product: coordinates, tiles and the rows of all groups are counted in 32 bits, and
// a sum is of `sum` values at most.
bool sizes_ok(int64_t rows, int64_t groups, int64_t n, int64_t k, int64_t sum) {
  if (rows < 0 || groups < 0 || n < 0 || k < 0 || rows > kMaxI32 - 4096 || n > kMaxI32 - 4096 ||
      k > kMaxI32 - 4096 || groups > nvfp4::kMatmulMaxGroups || groups * n > kMaxI32 - 4096 ||
      sum > nvfp4::kMatmulMaxSum)
    return false;
  return true;
}
bool tiles_ok(int64_t tiles) { return tiles <= (1 << 26); }

nvfp4_status check_ws(const void* workspace, size_t ws_bytes) {
  if (!workspace) return NVFP4_ERR_NULL;
  if (ws_bytes < nvfp4::kMatmulWsBytes) return NVFP4_ERR_SHAPE;
  return aligned(workspace, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}
void fill_ws(nvfp4::MatmulParams& p, void* workspace) {
  uint8_t* at = static_cast<uint8_t*>(workspace);
  p.tickets = reinterpret_cast<uint32_t*>(at);
  at += nvfp4::kMatmulTicketBytes;
  p.part = reinterpret_cast<float*>(at);
  p.padded = at + (size_t)4 * nvfp4::kMatmulMaxCtas * nvfp4::kMatmulPart;
}

// What the two products over ragged rows have in common.
nvfp4_status check_rows_product(const uint8_t* a_codes, const uint8_t* a_scales,
                                const uint8_t* b_codes, const uint8_t* b_scales, int64_t groups,
                                const int32_t* group_start, const void* out, const void* workspace,
                                size_t ws_bytes, const int32_t* status) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !out || (groups > 1 && !group_start))
    return NVFP4_ERR_NULL;
  const nvfp4_status e = check_ws(workspace, ws_bytes);
  if (e != NVFP4_OK) return e;
  for (const void* q : {(const void*)a_codes, (const void*)a_scales, (const void*)b_codes,
                        (const void*)b_scales, out})
    if (!aligned(q, 16)) return NVFP4_ERR_ALIGN;
  return aligned(group_start, 4) && aligned(status, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

}  // namespace

extern "C" {

size_t nvfp4_grouped_matmul_ws_bytes(void) { return nvfp4::kMatmulWsBytes; }

nvfp4_status nvfp4_grouped_matmul(const nvfp4_operand* a, const nvfp4_operand* b, int64_t rows,
                                  int64_t groups, int64_t out_cols, int64_t cols,
                                  const int32_t* group_start, void* out, void* workspace,
                                  size_t ws_bytes, int32_t* status, void* stream) {
  if (!a || !b) return NVFP4_ERR_NULL;
  if (!sizes_ok(rows, groups, out_cols, cols, cols) || cols % 32 != 0 ||
      !tiles_ok((rows / 256 + groups + 1) * (out_cols / 128 + 1)))
    return NVFP4_ERR_SHAPE;
  for (const nvfp4_operand* o : {a, b})
    if (!(o->scale_max >= 0.0f) || !std::isfinite(o->scale_max)) return NVFP4_ERR_ENUM;
  if (a->amax_count != 1 && a->amax_count != rows) return NVFP4_ERR_SHAPE;
  if (b->amax_count != groups) return NVFP4_ERR_SHAPE;
  if (rows == 0 || groups == 0 || out_cols == 0) return NVFP4_OK;
  if (cols == 0) return NVFP4_ERR_SHAPE;
  if (!a->amax || !b->amax) return NVFP4_ERR_NULL;
  const nvfp4_status e =
      check_rows_product(a->codes, a->scales, b->codes, b->scales, groups, group_start, out,
                         workspace, ws_bytes, status);
  if (e != NVFP4_OK) return e;
  if (!aligned(a->amax, 4) || !aligned(b->amax, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::MatmulParams p{};
  p.f_sf = b->scales;
  p.c_sf = a->scales;
  p.f_rows = groups * out_cols;
  p.c_rows = rows;
  p.sf_stride = cols / 16;
  p.N = (int32_t)out_cols;
  p.K = cols;
  p.E = (int32_t)groups;
  p.start = group_start;
  p.c_amax = a->amax;
  p.f_amax = b->amax;
  p.c_amax_each = a->amax_count == rows && rows > 1;
  p.c_M = a->scale_max > 0.0f ? a->scale_max : 448.0f;
  p.f_M = b->scale_max > 0.0f ? b->scale_max : 448.0f;
  p.out = out;
  p.status = status;
  fill_ws(p, workspace);
  return cuda_status(nvfp4::launch_matmul(nvfp4::kMatmulNvfp4, p, b->codes, a->codes,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_mx_grouped_matmul(const uint8_t* a_codes, const uint8_t* a_scales,
                                     const uint8_t* b_codes, const uint8_t* b_scales, int64_t rows,
                                     int64_t groups, int64_t out_cols, int64_t cols,
                                     const int32_t* group_start, void* out, void* workspace,
                                     size_t ws_bytes, int32_t* status, void* stream) {
  if (!sizes_ok(rows, groups, out_cols, cols, cols) || cols % 32 != 0 ||
      !tiles_ok((rows / 256 + groups + 1) * (out_cols / 128 + 1)))
    return NVFP4_ERR_SHAPE;
  if (rows == 0 || groups == 0 || out_cols == 0) return NVFP4_OK;
  if (cols == 0) return NVFP4_ERR_SHAPE;
  const nvfp4_status e = check_rows_product(a_codes, a_scales, b_codes, b_scales, groups,
                                            group_start, out, workspace, ws_bytes, status);
  if (e != NVFP4_OK) return e;
  nvfp4::MatmulParams p{};
  p.f_sf = b_scales;
  p.c_sf = a_scales;
  p.f_rows = groups * out_cols;
  p.c_rows = rows;
  p.sf_stride = cols / 32;
  p.N = (int32_t)out_cols;
  p.K = cols;
  p.E = (int32_t)groups;
  p.start = group_start;
  p.out = out;
  p.status = status;
  fill_ws(p, workspace);
  return cuda_status(nvfp4::launch_matmul(nvfp4::kMatmulMx, p, b_codes, a_codes,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_mx_grouped_wgrad(const uint8_t* g_codes, const uint8_t* g_scales,
                                    const uint8_t* x_codes, const uint8_t* x_scales, int64_t rows,
                                    int64_t groups, int64_t out_rows, int64_t out_cols,
                                    const int32_t* group_start, void* out, int32_t out_fp32,
                                    void* workspace, size_t ws_bytes, int32_t* status,
                                    void* stream) {
  if (!sizes_ok(rows, groups, out_rows, out_cols, rows) || rows % 32 != 0 ||
      !tiles_ok(groups * (out_rows / 256 + 1) * (out_cols / 128 + 1)))
    return NVFP4_ERR_SHAPE;
  if (out_fp32 != 0 && out_fp32 != 1) return NVFP4_ERR_ENUM;
  if (groups == 0 || out_rows == 0 || out_cols == 0) return NVFP4_OK;
  if (!out || (groups > 1 && !group_start) ||
      (rows > 0 && (!g_codes || !g_scales || !x_codes || !x_scales)))
    return NVFP4_ERR_NULL;
  const nvfp4_status e = check_ws(workspace, ws_bytes);
  if (e != NVFP4_OK) return e;
  for (const void* q : {(const void*)g_codes, (const void*)g_scales, (const void*)x_codes,
                        (const void*)x_scales, (const void*)out})
    if (!aligned(q, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(group_start, 4) || !aligned(status, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::MatmulParams p{};
  // The product's lanes are features. With g's rows there a lane holds a piece of a result's row
  // of bf16, which leaves by tensor map where rows are whole 32 bytes; else x's rows, whose lanes
  // hold neighbours. (Not by out's address: the two are cut differently, and the order of a sum
  // depends on the sizes alone.)
  p.turn = !out_fp32 && out_cols % 16 == 0;
  p.f_sf = p.turn ? g_scales : x_scales;
  p.c_sf = p.turn ? x_scales : g_scales;
  p.f_rows = p.turn ? out_rows : out_cols;
  p.c_rows = p.turn ? out_cols : out_rows;
  p.sf_stride = rows / 32;
  p.N = (int32_t)p.f_rows;
  p.C = (int32_t)p.c_rows;
  p.K = rows;
  p.E = (int32_t)groups;
  p.start = group_start;
  p.out = out;
  p.out_f32 = out_fp32;
  p.status = status;
  fill_ws(p, workspace);
  return cuda_status(nvfp4::launch_matmul(nvfp4::kMatmulMxWgrad, p,
                                          p.turn ? g_codes : x_codes, p.turn ? x_codes : g_codes,
                                          static_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_add_rms_norm(const nvfp4_config* cfg, int32_t target, const void* x,
                                const void* residual, const void* weight, int64_t rows,
                                int64_t cols, float eps, void* h, void* y,
                                const float* global_amax, float* row_amax, const nvfp4_out* out,
                                int32_t* status, void* stream) {
  if (!cfg) return NVFP4_ERR_NULL;
  const bool fp4 = target == NVFP4_TARGET_NVFP4;
  if ((!fp4 && target != NVFP4_TARGET_MXFP8) || !(eps >= 0.0f) || !std::isfinite(eps) ||
      cfg->blocks != NVFP4_BLOCKS_ROW || cfg->rounding != NVFP4_ROUND_RNE)
    return NVFP4_ERR_ENUM;
  if (fp4 && (cfg->scale_fmt != NVFP4_SCALE_E4M3 || !(cfg->scale_max >= 0.0f) ||
              !std::isfinite(cfg->scale_max) ||
              (cfg->four_over_six != 0 && cfg->four_over_six != 1) ||
              (cfg->four_over_six && cfg->four_over_six_rule != NVFP4_FOS_MSE)))
    return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || rows > kMaxI32 || cols > nvfp4::kNormMaxCols ||
      cols % (fp4 ? 16 : 32) != 0)
    return NVFP4_ERR_SHAPE;
  if (rows == 0 || cols == 0) return NVFP4_OK;
  if (!x || !weight || !out || !out->codes || !out->scales || (residual && !h) ||
      (fp4 && !global_amax && !row_amax))
    return NVFP4_ERR_NULL;
  if (!fp4 && out->dequant) return NVFP4_ERR_ENUM;
  for (const void* q : {x, residual, weight, (const void*)h, (const void*)y,
                        (const void*)out->codes, (const void*)out->scales,
                        (const void*)out->choice, (const void*)out->dequant})
    if (!aligned(q, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(global_amax, 4) || !aligned(row_amax, 4) || !aligned(status, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::NormParams p{};
  p.x = static_cast<const uint4*>(x);
  p.res = static_cast<const uint4*>(residual);
  p.w = static_cast<const uint4*>(weight);
  p.R = rows;
  p.C = (int32_t)cols;
  p.eps = eps;
  p.h = static_cast<uint4*>(h);
  p.y = static_cast<uint4*>(y);
  p.gamax = fp4 ? global_amax : nullptr;
  p.M = cfg->scale_max > 0.0f ? cfg->scale_max : cfg->four_over_six ? 256.0f : 448.0f;
  p.row_amax = row_amax;
  p.codes = out->codes;
  p.scales = out->scales;
  p.choice = cfg->four_over_six ? out->choice : nullptr;
  p.dq = static_cast<uint4*>(out->dequant);
  p.status = status;
  return cuda_status(nvfp4::launch_norm(p, fp4 ? 1 : 0, fp4 && cfg->four_over_six != 0,
                                        static_cast<cudaStream_t>(stream)));
}

size_t nvfp4_add_rms_norm_ws_bytes(void) { return nvfp4::kNormWsBytes; }

nvfp4_status nvfp4_add_rms_norm_bwd(const void* gy, const void* h, const void* weight,
                                    const void* gh, int64_t rows, int64_t cols, float eps,
                                    void* gx, float* gw, void* workspace, size_t ws_bytes,
                                    int32_t* status, void* stream) {
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return NVFP4_ERR_ENUM;
  if (rows < 0 || cols < 0 || rows > kMaxI32 || cols > nvfp4::kNormMaxCols || cols % 16 != 0)
    return NVFP4_ERR_SHAPE;
  if (cols == 0) return NVFP4_OK;
  if (!gw) return NVFP4_ERR_NULL;
  if (!aligned(gw, 16)) return NVFP4_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0)  // a sum over nothing
    return cuda_status(nvfp4::launch_zero_words(reinterpret_cast<uint32_t*>(gw), cols, st));
  if (!gy || !h || !weight || !gx || !workspace) return NVFP4_ERR_NULL;
  if (ws_bytes < nvfp4::kNormWsBytes) return NVFP4_ERR_SHAPE;
  for (const void* q : {gy, h, weight, gh, (const void*)gx, (const void*)workspace})
    if (!aligned(q, 16)) return NVFP4_ERR_ALIGN;
  if (!aligned(status, 4)) return NVFP4_ERR_ALIGN;
  nvfp4::NormBwdParams p{};
  p.gy = static_cast<const uint4*>(gy);
  p.h = static_cast<const uint4*>(h);
  p.w = static_cast<const uint4*>(weight);
  p.gh = static_cast<const uint4*>(gh);
  p.R = rows;
  p.C = (int32_t)cols;
  p.eps = eps;
  p.gx = static_cast<uint4*>(gx);
  p.gw = gw;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  return cuda_status(nvfp4::launch_norm_bwd(p, st));
}

}  // extern "C"
