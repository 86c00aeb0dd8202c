// kv_append.cu -- K and V rows quantised into the paged NVFP4 cache.
//
// The encoding is the row encoding of nvfp4_quantize with one slice per KV
// head: a lane holds 8 values (one 128-bit load), two adjacent lanes a block
// of 16. Each head has its own outer scale, so d = dec(code) g and 1/d are
// computed for the block instead of read from a per-slice table. A thread keeps
// its place in the heads and takes several tokens, kBatch loads at a time, so that
// the head's constants (a division, two reciprocals) are worked out once. Bound by
// DRAM and issue together: 2 bytes read, 0.5625 (+ 2 with the de-quantised rows) written
// per value, and the encoder's instructions keep 77% of the issue slots busy. 16381
// tokens of 8 heads of 128 with de-quantised rows: 30.1 us, 5.08 TB/s (75% of the
// measured copy rate), without 26.7 us (48%: the same instructions, fewer bytes), with 4/6
// 41.6 and 39.5 us; one token of 48 requests: 2.0 us.
#include "encode.cuh"
#include "kv.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

constexpr int kBatch = 4;

// Block (x, side, z): tokens x * per .. + per - 1 of K or V, lanes z * 256 .. of a
// token's W = heads * LPH; `rows` tokens side by side in a block.
template <int LPH, bool FOS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendParams p,
                                                             const FastDiv by_page,
                                                             const int rows,
                                                             const FastDiv by_lanes,
                                                             const int per) {
  pdl_begin();
  const int side = blockIdx.y;
  const int W = p.H * LPH, w0 = blockIdx.z * kThreads, lanes = min(W - w0, kThreads);
  // threads past the last whole row follow another one's, so that warps stay whole
  const int r0 = (int)fastdiv(threadIdx.x, by_lanes);
  const bool mine = r0 < rows && (int)threadIdx.x - r0 * lanes < lanes;
  const int wl = w0 + (mine ? (int)threadIdx.x - r0 * lanes : (int)(threadIdx.x & 7));
  const int row = mine ? r0 : 0;
  const int h = wl / LPH, l = wl % LPH;
  const int64_t first = (int64_t)blockIdx.x * per, last = min(first + per, p.T);
  const SliceScale ss = slice_scale(p.amax[side][h], p.M);
  if (ss.bad) flag(p.status, NVFP4_DEV_BAD_AMAX_BIT);
  const DirectScales<0> scales{ss.g};
  const uint16_t* src = p.x[side] + wl * 8;
  uint32_t* codes = reinterpret_cast<uint32_t*>(p.codes[side]);

  for (int64_t t0 = first; t0 < last; t0 += kBatch * rows) {
    uint4 raw[kBatch];
    int64_t slot[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t t = min(t0 + u * rows + row, last - 1);
      raw[u] = __ldcs(reinterpret_cast<const uint4*>(src + t * p.st[side]));
      slot[u] = p.slots[t];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int64_t t = t0 + u * rows + row;
      if (t0 + u * rows >= last) break;
      const bool ok = mine && t < last;
      f2 x[4];
      unpack8(raw[u], x);
      uint32_t m = absmax_bits4(raw[u]);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      if (m >= 0x7F80u) flag(p.status, NVFP4_DEV_NONFINITE_INPUT_BIT);

      const float amax = __uint_as_float(m << 16);
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
      if (!ok) continue;
      if (p.dq[side]) __stcs(p.dq[side] + t * W + wl, dq);
      if (slot[u] < 0 || slot[u] >= p.n_slots) {
        if (slot[u] != -1) flag(p.status, kDevBadIndex);
        continue;
      }
      int64_t page, off;
      if (p.n_slots <= 0xFFFFFFFFll) {
        page = fastdiv((uint32_t)slot[u], by_page);
        off = slot[u] - page * p.P;
      } else {
        page = slot[u] / p.P;
        off = slot[u] % p.P;
      }
      const int64_t at = ((page * p.H + h) * p.P + off) * LPH + l;
      codes[at] = code;
      if ((l & 1) == 0) p.scales[side][at >> 1] = (uint8_t)sc;
    }
  }
}

template <int LPH, bool FOS>
cudaError_t launch_t(const KvAppendParams& p, cudaStream_t st) {
  const int64_t W = (int64_t)p.H * LPH;
  const int64_t chunks = (W + kThreads - 1) / kThreads;
  const int lanes = (int)std::min<int64_t>(W, kThreads), rows = kThreads / lanes;
  // tokens per CTA: four batches where that still leaves two waves of CTAs
  int64_t per = 4 * kBatch * rows;
  while (per > rows && (p.T + per - 1) / per * 2 * chunks < (int64_t)sm_count() * 16) per /= 2;
  per = std::max<int64_t>(per, rows);
  const int64_t ctas = (p.T + per - 1) / per;
  if (ctas > INT32_MAX || chunks > 65535) return cudaErrorInvalidValue;
  return launch_pdl(kv_append_kernel<LPH, FOS>, dim3((unsigned)ctas, 2, (unsigned)chunks),
                    dim3(kThreads), st, p, make_fastdiv((uint32_t)p.P), rows,
                    make_fastdiv((uint32_t)lanes), (int)per);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int D, bool fos, cudaStream_t st) {
  if (D == 128) return fos ? launch_t<16, true>(p, st) : launch_t<16, false>(p, st);
  return fos ? launch_t<8, true>(p, st) : launch_t<8, false>(p, st);
}

}  // namespace nvfp4
