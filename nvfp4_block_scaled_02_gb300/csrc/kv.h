// kv.h -- internal host-side interface between the C ABI of the KV-cache
// operators (api_kv.cu) and their kernels. Not installed; the public interface
// is nvfp4.h.
#pragma once
#include <atomic>

#include "launch.h"

namespace nvfp4 {

constexpr int kDevBadIndex = NVFP4_DEV_BAD_INDEX;
constexpr int kDevNoPages = NVFP4_DEV_NO_PAGES;
constexpr int kDevTimeout = NVFP4_DEV_TIMEOUT;

// launch_pdl with dynamic shared memory.
template <class... KArgs, class... Args>
cudaError_t launch_pdl_smem(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, static_cast<Args&&>(args)...);
}

// Lets `kernel` use `smem` bytes of dynamic shared memory on the current device;
// `ready` keeps a bit per device, so that only a device's first call sets it.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, size_t smem, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Block tables and slot maps.
struct KvPlanParams {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t B;
  int32_t* table;
  int32_t cols;
  FastDiv by_page;
  int32_t P;
  const int32_t* free_pages;
  int32_t n_free;
  int32_t T;
  int32_t* seq_len;
  int32_t* q_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* used;
  int32_t* status;
};
cudaError_t launch_kv_plan(const KvPlanParams& p, cudaStream_t st);

// Head norms and rotation. Rows: bf16, token t of tensor x at x + t * stride.
struct QkRopeParams {
  int64_t T;
  int32_t hq, hk, R;
  float eps;
  const uint4* qw;         // bf16 [D] or null
  const uint4* kw;
  const int32_t* pos;
  const float* cs;         // [max_pos][R]
  int64_t max_pos;
  const uint16_t *q, *k;   // inputs of the forward
  int64_t q_st, k_st;
  uint16_t *qo, *ko;       // forward: outputs; backward: gq, gk
  int64_t qo_st, ko_st;
  const uint16_t *gq, *gk; // backward: gradients of the outputs
  int64_t gq_st, gk_st;
  float *gqw, *gkw;        // backward: weight gradients or null
  float* ws;               // backward: partial sums, then the ticket word
  int32_t* status;
};
constexpr int kQkMaxCtas = 1024;                        // CTAs of the backward at most
constexpr size_t kQkWsBytes = (size_t)kQkMaxCtas * 2 * 128 * 4 + 16;
cudaError_t launch_qk_rope(const QkRopeParams& p, int D, bool interleaved, cudaStream_t st);
cudaError_t launch_qk_rope_bwd(const QkRopeParams& p, int D, bool interleaved, cudaStream_t st);

// K and V rows into the cache.
struct KvAppendParams {
  const uint16_t* x[2];    // K, V
  int64_t st[2];
  uint8_t* codes[2];
  uint8_t* scales[2];
  const float* amax[2];
  uint4* dq[2];            // or null
  const int64_t* slots;
  int64_t T, n_slots;
  int32_t H, P;
  float M;
  int32_t* status;
};
cudaError_t launch_kv_append(const KvAppendParams& p, int D, bool fos, cudaStream_t st);

// Attention over the cache.
struct KvAttnParams {
  const uint8_t *kc, *ks, *vc, *vs;
  const float *k_amax, *v_amax;
  float M;
  int64_t pages;
  int32_t hk, P, page_shift;  // page_shift: log2(P) or -1
  FastDiv by_page, by_group;
  const int32_t *table, *seq_len, *q_start;
  int32_t B, cols, T, hq, G, max_q, window;
  float scale;
  const uint16_t* q;
  int64_t q_st;
  uint16_t* out;
  float* lse;
  int32_t few_rows;        // requests with at most so many rows per KV head go to kv_attn.cu
  int32_t over_rows;       // ... those with more than so many, in one launch of it
  uint32_t* tickets;       // [kAttnTickets], zero between calls
  float* part;             // partial results, two records per CTA
  int32_t* status;
};
constexpr int kAttnMaxCtas = 1024;
constexpr int kAttnRows = 16;                           // query rows of an item at most
constexpr int kAttnRecord = kAttnRows * (128 + 2);      // floats: rows x (out, max, sum)
constexpr int kPrefillMaxCtas = 192;
constexpr int kPrefillRecord = 256 * (128 + 2);
constexpr int kAttnTickets = kAttnMaxCtas + 8 * kPrefillMaxCtas;
// the two kernels of a call run one after the other: they share the records
constexpr size_t kAttnPartBytes =
    (size_t)4 * std::max(2 * kAttnMaxCtas * kAttnRecord, 2 * kPrefillMaxCtas * kPrefillRecord);
constexpr size_t kAttnWsBytes = (size_t)4 * kAttnTickets + kAttnPartBytes;
cudaError_t launch_kv_few(KvAttnParams p, int D, cudaStream_t st);
cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, cudaStream_t st);

}  // namespace nvfp4
