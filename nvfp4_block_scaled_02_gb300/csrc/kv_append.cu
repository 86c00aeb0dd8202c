// kv_append.cu -- K and V rows quantised into the paged NVFP4 cache.
//
// The encoding is the row encoding of nvfp4_quantize with one slice per KV
// head: a lane holds 8 values (one 128-bit load), two adjacent lanes a block
// of 16. Each head has its own outer scale, so d = dec(code) g and 1/d are
// computed for the block instead of read from a per-slice table. Bound by
// DRAM: 2 bytes read, 0.5625 (+ 2 with the de-quantised rows) written per
// value.
#include "encode.cuh"
#include "kv.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

template <int LPH, bool FOS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p,
                                                             FastDiv by_page) {
  pdl_begin();
  const int side = blockIdx.y;
  const int W = p.H * LPH;  // lanes of one token, a multiple of 8
  const int64_t n = p.T * W;
  const int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const bool ok = i0 < n;
  const int64_t i = ok ? i0 : n - 1;  // the last warp stays whole for the shuffles
  const int64_t t = i / W;
  const int wl = (int)(i - t * W), h = wl / LPH, l = wl % LPH;
  const SliceScale ss = slice_scale(p.amax[side][h], p.M);
  if (ss.bad) flag(p.status, NVFP4_DEV_BAD_AMAX_BIT);
  const uint4 v = *reinterpret_cast<const uint4*>(p.x[side] + t * p.st[side] + wl * 8);
  f2 x[4];
  unpack8(v, x);
  uint32_t m = absmax_bits4(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  if (m >= 0x7F80u) flag(p.status, NVFP4_DEV_NONFINITE_INPUT_BIT);

  const float amax = __uint_as_float(m << 16);
  const DirectScales<0> scales{ss.g};
  const uint4 rb = make_uint4(0, 0, 0, 0);
  uint32_t c6, c4 = 0;
  if constexpr (FOS) {
    const uint32_t cc = scale_encode2<0>(__fmul_rn(amax, ss.rden6), __fmul_rn(amax, ss.rden4));
    c6 = cc & 0xFFu;
    c4 = cc >> 8;
  } else {
    c6 = scale_encode<0>(__fmul_rn(amax, ss.rden6));
  }
  float d6, inv6;
  scales(c6, d6, inv6);
  f2 v6[4];
  uint32_t code = cand8<false>(x, inv6, rb, 0u, true, v6);
  uint32_t sc = c6;
  uint4 dq = dequant8(v6, d6);
  if constexpr (FOS) {
    float d4, inv4;
    scales(c4, d4, inv4);
    f2 v4[4];
    const uint32_t q4 = cand8<false>(x, inv4, rb, 0u, true, v4);
    const float h6 = half_metric_q(x, v6, d6, 0), h4 = half_metric_q(x, v4, d4, 0);
    const float e6 = combine_halves(h6, __shfl_xor_sync(0xFFFFFFFFu, h6, 1), 0);
    const float e4 = combine_halves(h4, __shfl_xor_sync(0xFFFFFFFFu, h4, 1), 0);
    const bool pick4 = e4 < e6;
    code = pick4 ? q4 : code;
    sc = pick4 ? c4 : c6;
    dq = dequant8_pick(v4, v6, pick4, d4, d6);
  }
  if (!ok) return;
  if (p.dq[side]) __stcs(p.dq[side] + i, dq);
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) {
    if (slot != -1) flag(p.status, kDevBadIndex);
    return;
  }
  int64_t page, off;
  if (p.n_slots <= 0xFFFFFFFFll) {
    page = fastdiv((uint32_t)slot, by_page);
    off = slot - page * p.P;
  } else {
    page = slot / p.P;
    off = slot % p.P;
  }
  const int64_t row = (page * p.H + h) * p.P + off;
  reinterpret_cast<uint32_t*>(p.codes[side])[row * LPH + l] = code;
  if ((l & 1) == 0) p.scales[side][(row * LPH + l) >> 1] = (uint8_t)sc;
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int D, bool fos, cudaStream_t st) {
  const int64_t ctas = (p.T * p.H * (D / 8) + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas, 2);
  const FastDiv by_page = make_fastdiv((uint32_t)p.P);
  if (D == 128)
    return fos ? launch_pdl(kv_append_kernel<16, true>, grid, dim3(kThreads), st, p, by_page)
               : launch_pdl(kv_append_kernel<16, false>, grid, dim3(kThreads), st, p, by_page);
  return fos ? launch_pdl(kv_append_kernel<8, true>, grid, dim3(kThreads), st, p, by_page)
             : launch_pdl(kv_append_kernel<8, false>, grid, dim3(kThreads), st, p, by_page);
}

}  // namespace nvfp4
