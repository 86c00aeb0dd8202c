// norm.cu -- the residual's addition, the RMS norm of a token and its encoding in
// MXFP8 or NVFP4 in one pass, and the norm's gradient.
//
// With h = bf16(x + residual) and r = 1 / sqrt(mean(h^2) + eps), a row's output is
// y = h r w. One CTA per row at a time; a thread keeps blocks of 16 values of the
// row in registers, so that everything is read once.
//
// With an outer scale for each row, r is left out of the codes: the encoding of
// y / r = h w, whose products of two bf16 are exact in fp32, has y's codes and
// block scales, and r goes into the row's amax. The codes then do not depend on
// the order of the sum of squares.
//
// Both passes are bound by DRAM: 8192 x 4096 with a residual, in MXFP8, 37 us
// (94% of the measured copy rate), the gradient 47 us (84%; 32768 rows 96%: about
// 8 us do not depend on the rows, 3 of them the sum over CTAs in a launch of its
// own). To NVFP4 by row 40 us, by tensor 37; with Four-Over-Six, which encodes
// every block twice, 50 and 44. 32 rows take 2.6 us on the device, the call from
// Python 13 (7 with outputs passed in).
#include "encode.cuh"
#include "norm.h"
#include "tcgen05.cuh"

namespace nvfp4 {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMaxThreads = 512;

__device__ __forceinline__ float2 dot_add(float2 a, float2 acc) { return f2_fma(a, a, acc); }

// 8 bf16 sums, each rounded to bf16
__device__ __forceinline__ uint4 add8(uint4 a, uint4 b) {
  f2 u[4], v[4];
  unpack8(a, u);
  unpack8(b, v);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = pack_bf16x2(__fadd_rn(u[i].x, v[i].x), __fadd_rn(u[i].y, v[i].y));
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 pack8(const f2 (&v)[4]) {
  return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                    pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
}
__device__ __forceinline__ float nan32() { return __uint_as_float(0x7FFFFFFFu); }
// The largest magnitude; with NANS, NaN if one is.
template <bool NANS>
__device__ __forceinline__ float absmax8(const f2 (&v)[4], float m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fabsf(v[i].x), b = fabsf(v[i].y);
    if constexpr (NANS) asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(a), "f"(b));
    else m = fmax3(m, a, b);
  }
  return m;
}
// 1 / sqrt(mean + eps); 0 for a row of zeros without eps, NaN where the sum is no finite number
// (NaN or infinite values, squares past fp32), so that the row's results show it
__device__ __forceinline__ float inv_rms(float sum, int C, float eps) {
  const float m = __fadd_rn(__fdiv_rn(sum, (float)C), eps);
  if (!(m <= kFltMax)) return nan32();
  return m > 0.0f ? rsqrtf(m) : 0.0f;
}

enum { kMx = 0, kRow = 1, kTensor = 2 };  // MXFP8, NVFP4 by row, NVFP4 by tensor

template <int MODE, bool FOS, int K>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NormParams p) {
  pdl_begin();
  __shared__ float s_sum[2][kMaxThreads / 32], s_max[2][kMaxThreads / 32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int blocks = p.C / 16;
  auto load_row = [&](int64_t row, uint4 (&x)[K][2], uint4 (&r)[K][2]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = k * nt + tid;
      const bool ok = row < p.R && b < blocks;
      const int64_t at = (row * blocks + b) * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[k][i] = ok ? __ldcs(p.x + at + i) : make_uint4(0, 0, 0, 0);
        if (p.res) r[k][i] = ok ? __ldcs(p.res + at + i) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  uint4 wt[K][2];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = k * nt + tid;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      wt[k][i] = b < blocks ? __ldg(p.w + 2 * b + i) : make_uint4(0, 0, 0, 0);
  }
  SliceScale st{};
  if constexpr (MODE == kTensor) {
    st = slice_scale(p.gamax[0], p.M);
    if (st.bad && blockIdx.x == 0 && tid == 0) flag(p.status, NVFP4_DEV_BAD_AMAX);
  }
  uint4 x[K][2], res[K][2];
  load_row(blockIdx.x, x, res);
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x, par ^= 1) {
    uint4 h[K][2];
    float m = 0.0f;
    f2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = k * nt + tid;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[k][i] = x[k][i];
        if (p.res) {
          h[k][i] = add8(x[k][i], res[k][i]);
          if (b < blocks) __stcs(p.h + (row * blocks + b) * 2 + i, h[k][i]);
        }
        f2 v[4];
        unpack8(h[k][i], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = dot_add(v[j], acc);
        if constexpr (MODE == kRow) {
          f2 w[4];
          unpack8(wt[k][i], w);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = f2_mul(v[j], w[j]);
          m = absmax8<true>(v, m);
        }
      }
    }
    load_row(row + gridDim.x, x, res);  // the next row in flight while this one is encoded
    float sum = __fadd_rn(acc.x, acc.y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kAll, sum, d));
    if constexpr (MODE == kRow)
      m = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(m)));
    if (lane == 0) {
      s_sum[par][warp] = sum;
      s_max[par][warp] = m;
    }
    __syncthreads();
    sum = s_sum[par][0];
    m = s_max[par][0];
    for (int i = 1; i < warps; ++i) {
      sum = __fadd_rn(sum, s_sum[par][i]);
      m = __uint_as_float(max(__float_as_uint(m), __float_as_uint(s_max[par][i])));
    }
    const float r = inv_rms(sum, p.C, p.eps);
    SliceScale ss = st;
    float g = 0.0f;  // of the values that the codes stand for
    bool bad = r != r;
    if constexpr (MODE == kRow) {
      bad = bad || !(m <= kFltMax);
      ss = slice_scale(m, p.M);
      // (r m may be too small for 32 bits where m is not 0: then the row's values are 0)
      const float top =
          bad ? nan32() : m > 0.0f ? fmaxf(__fmul_rn(m, r), __uint_as_float(1u)) : 0.0f;
      g = slice_scale(top, p.M).g;
      if (tid == 0) p.row_amax[row] = top;
    } else {
      g = ss.g;
    }
    if (tid == 0 && bad) flag(p.status, NVFP4_DEV_NONFINITE_INPUT);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int b = k * nt + tid;
      const bool ok = b < blocks;
      const int64_t at = row * blocks + b;
      f2 v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f2 w[4];
        unpack8(h[k][i], v[i]);
        unpack8(wt[k][i], w);
        if constexpr (MODE == kRow) {
          if (p.y) {
            f2 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = f2_mul(f2_mul(v[i][j], make_float2(r, r)), w[j]);
            if (ok) __stcs(p.y + 2 * at + i, pack8(y));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(v[i][j], w[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = f2_mul(f2_mul(v[i][j], make_float2(r, r)), w[j]);
          if (p.y && ok) __stcs(p.y + 2 * at + i, pack8(v[i]));
        }
      }
      float bm = absmax8<true>(v[1], absmax8<true>(v[0], 0.0f));
      // A NVFP4 block with a value that is no finite number gets a NaN for its scale and codes of 0
      // (nvfp4_requant_transpose knows no NaN scales); an MXFP8 code can be NaN, and infinities
      // saturate.
      if (!(bm <= kFltMax)) {
        flag(p.status, NVFP4_DEV_NONFINITE_INPUT);
        bm = MODE == kMx ? absmax8<false>(v[1], absmax8<false>(v[0], 0.0f)) : nan32();
      }
      if (MODE != kMx && bad) bm = nan32();
      if constexpr (MODE == kMx) {
        // the block of 32 is this thread's 16 values and its neighbour's
        bm = fmaxf(bm, __shfl_xor_sync(kAll, bm, 1));
        const int e = mx_shared_exp(bm);
        const float sc = exp2_neg(e);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 a = v[i / 2][i % 2 * 2], bb = v[i / 2][i % 2 * 2 + 1];
          c[i] = e4m3x4_rn(__fmul_rn(a.x, sc), __fmul_rn(a.y, sc), __fmul_rn(bb.x, sc),
                           __fmul_rn(bb.y, sc));
        }
        if (ok) {
          __stcs(reinterpret_cast<uint4*>(p.codes) + at, make_uint4(c[0], c[1], c[2], c[3]));
          if (!(tid & 1)) p.scales[at >> 1] = (uint8_t)(e + 127);
        }
      } else {
        const uint4 none = make_uint4(0, 0, 0, 0);
        BlockResult q = encode_block_f<0, false, FOS>(v[0], v[1], bm, ss, DirectScales<0>{ss.g},
                                                      none, none, false);
        if (bm != bm) q.codes[0] = q.codes[1] = 0;
        if (ok) {
          __stcs(reinterpret_cast<uint2*>(p.codes) + at, make_uint2(q.codes[0], q.codes[1]));
          p.scales[at] = (uint8_t)q.scale;
          if (p.dq) {
            const float d = bm == bm ? __fmul_rn(e4m3_value(q.scale), g) : bm;
            f2 t[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              e2m1x8_to_f2(q.codes[i], t);
              __stcs(p.dq + 2 * at + i, dequant8(t, d));
            }
          }
        }
        if constexpr (FOS) {
          if (p.choice) {
            const uint32_t word = __ballot_sync(kAll, ok && q.pick4);
            const int wi = k * warps + warp, words = (blocks + 31) / 32;
            if (lane == 0 && wi < words) p.choice[row * words + wi] = word;
          }
        }
      }
    }
  }
}

// Gradient. u = gy w: gx = r (u - h r^2 mean(u h)) + gh, and the weight's gradient is the
// sum over rows of gy h r. Rows come by bulk copies into a ring in shared memory, so that
// several are on their way whatever the registers hold (8192 x 4096: 58 us with the next row
// in registers, 48 so); a thread keeps the weight gradients of its values over the CTA's rows,
// and a second kernel adds the CTAs' sums in order. Two rows between two barriers took 58 us.
constexpr long long kWaitCycles = 2000000000;  // about a second
constexpr int kMaxDepth = 8;
constexpr int kRingBwd = 200 * 1024;  // bytes of shared memory for rows on an SM

template <int K>
__global__ void __launch_bounds__(kMaxThreads, K == 1 ? 2 : 1)
norm_bwd_kernel(const NormBwdParams p, const int depth) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kMaxDepth];
  __shared__ float2 s_sum[2][kMaxThreads / 32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const int chunks = p.C / 8;
  const uint32_t bytes = (uint32_t)p.C * 2;  // of a row of one tensor
  if (tid == 0) {
    for (int i = 0; i < depth; ++i) mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_begin();
  __syncthreads();
  auto copy_row = [&](int64_t row, int slot) {  // one thread
    if (row >= p.R) return;
    uint8_t* to = ring + (size_t)slot * 3 * bytes;
    mbar_expect(&full[slot], p.gh ? 3 * bytes : 2 * bytes);
    const int64_t at = row * chunks;
    bulk_load(to, p.gy + at, bytes, &full[slot]);
    bulk_load(to + bytes, p.h + at, bytes, &full[slot]);
    if (p.gh) bulk_load(to + 2 * bytes, p.gh + at, bytes, &full[slot]);
  };
  if (tid == 0)
    for (int i = 0; i < depth; ++i) copy_row(blockIdx.x + (int64_t)i * gridDim.x, i);
  uint4 wt[K];
  f2 gw[K][4];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * nt + tid;
    wt[k] = c < chunks ? __ldg(p.w + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) gw[k][j] = make_float2(0.0f, 0.0f);
  }
  int slot = 0, par = 0;
  uint32_t turn = 0;
  bool alive = true;
  for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x, par ^= 1) {
    if (alive && !mbar_try(&full[slot], turn)) {
      const long long t0 = clock64();
      while (!mbar_try(&full[slot], turn))
        if (clock64() - t0 > kWaitCycles) {
          flag(p.status, NVFP4_DEV_TIMEOUT);
          alive = false;  // nothing is waited for any more; the barriers are still met
          break;
        }
    }
    const uint4* from = reinterpret_cast<const uint4*>(ring + (size_t)slot * 3 * bytes);
    uint4 gy[K], h[K], gh[K];
    f2 a2 = make_float2(0.0f, 0.0f), ad = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * nt + tid;
      const bool ok = c < chunks;
      gy[k] = ok ? from[c] : make_uint4(0, 0, 0, 0);
      h[k] = ok ? from[chunks + c] : make_uint4(0, 0, 0, 0);
      gh[k] = ok && p.gh ? from[2 * chunks + c] : make_uint4(0, 0, 0, 0);
      f2 g[4], v[4], w[4];
      unpack8(gy[k], g);
      unpack8(h[k], v);
      unpack8(wt[k], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a2 = f2_fma(v[j], v[j], a2);
        ad = f2_fma(f2_mul(g[j], w[j]), v[j], ad);
      }
    }
    float2 sum = make_float2(__fadd_rn(a2.x, a2.y), __fadd_rn(ad.x, ad.y));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      sum.x = __fadd_rn(sum.x, __shfl_xor_sync(kAll, sum.x, d));
      sum.y = __fadd_rn(sum.y, __shfl_xor_sync(kAll, sum.y, d));
    }
    if (lane == 0) s_sum[par][warp] = sum;
    __syncthreads();  // sums in; the row is in registers
    if (tid == 0) copy_row(row + (int64_t)depth * gridDim.x, slot);
    if (++slot == depth) slot = 0, turn ^= 1;
    sum = s_sum[par][0];
    for (int i = 1; i < warps; ++i) {
      sum.x = __fadd_rn(sum.x, s_sum[par][i].x);
      sum.y = __fadd_rn(sum.y, s_sum[par][i].y);
    }
    if (tid == 0 && !(sum.x <= kFltMax && fabsf(sum.y) <= kFltMax))
      flag(p.status, NVFP4_DEV_NONFINITE_INPUT);
    const float r = inv_rms(sum.x, p.C, p.eps);
    // r (u - h r^2 m) = r u - (h r) (r m r): r^2 alone may be past fp32
    const float t = -__fmul_rn(__fmul_rn(__fdiv_rn(sum.y, (float)p.C), r), r);
    const f2 r2 = make_float2(r, r), t2 = make_float2(t, t);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      f2 g[4], v[4], w[4], q[4], o[4];
      unpack8(gy[k], g);
      unpack8(h[k], v);
      unpack8(wt[k], w);
      unpack8(gh[k], q);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 x = f2_mul(v[j], r2);
        gw[k][j] = f2_fma(g[j], x, gw[k][j]);
        o[j] = f2_fma(x, t2, f2_mul(f2_mul(g[j], w[j]), r2));
        if (p.gh) o[j] = make_float2(__fadd_rn(o[j].x, q[j].x), __fadd_rn(o[j].y, q[j].y));
      }
      const int c = k * nt + tid;
      if (c < chunks) __stcs(p.gx + row * chunks + c, pack8(o));
    }
  }
  if (!alive) {  // copies in flight land before the CTA ends
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000) {
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * nt + tid;
    if (c >= chunks) continue;
    float4* to = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.C) + 2 * c;
    to[0] = make_float4(gw[k][0].x, gw[k][0].y, gw[k][1].x, gw[k][1].y);
    to[1] = make_float4(gw[k][2].x, gw[k][2].y, gw[k][3].x, gw[k][3].y);
  }
}

// gw[c] = sum over n rows of part[.][c]: a CTA to 32 columns, its warps take rows in turn.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) column_sum_kernel(const float* part, int n, int C,
                                                                    float* gw) {
  pdl_begin();
  __shared__ float s[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < C)
#pragma unroll 8
    for (int i = warp; i < n; i += kSumWarps) v = __fadd_rn(v, __ldcg(part + (int64_t)i * C + c));
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) v = __fadd_rn(v, s[i][lane]);
    gw[c] = v;
  }
}

// CTAs of `kernel` with so many threads and bytes of shared memory on an SM; `fit` keeps the answer
// for just these.
template <class Kernel>
int ctas_per_sm(Kernel kernel, int threads, std::atomic<int>& fit, size_t smem = 0) {
  int n = fit.load(std::memory_order_relaxed);
  if (n == 0) {
    n = resident_ctas(kernel, threads, smem);
    fit.store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int MODE, bool FOS, int K>
cudaError_t run(const NormParams& p, int threads, cudaStream_t st) {
  static std::atomic<int> fit[kMaxThreads / 32 + 1];
  const int per_sm = ctas_per_sm(norm_kernel<MODE, FOS, K>, threads, fit[threads / 32]);
  const int64_t grid = std::min<int64_t>(p.R, (int64_t)sm_count() * per_sm);
  return launch_pdl(norm_kernel<MODE, FOS, K>, dim3((unsigned)grid), dim3(threads), st, p);
}
template <int MODE, bool FOS>
cudaError_t sized(const NormParams& p, cudaStream_t st) {
  const int blocks = p.C / 16;
  auto threads = [&](int k) { return ((blocks + k - 1) / k + 31) / 32 * 32; };
  if (blocks <= kMaxThreads) return run<MODE, FOS, 1>(p, threads(1), st);
  return run<MODE, FOS, 2>(p, threads(2), st);
}

template <int K>
cudaError_t run_bwd(const NormBwdParams& p, cudaStream_t st) {
  const int chunks = p.C / 8, threads = ((chunks + K - 1) / K + 31) / 32 * 32;
  // rows on their way: at least two, and up to 4096 values so many that a thread's share of
  // shared memory is that of 1024 threads on an SM
  const int row = 3 * 2 * p.C, room = K == 1 ? kRingBwd / 1024 * threads : kRingBwd;
  const int depth = std::max(2, std::min(kMaxDepth, room / row));
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(norm_bwd_kernel<K>, kRingBwd, ready);
  if (e != cudaSuccess) return e;
  // (by the width, which shared memory goes by: the grid decides how gw's sum is grouped, and the
  // same call has to give the same bits whatever was called before it)
  static std::atomic<int> fit[kNormMaxCols / 16 + 1];
  const int per_sm =
      ctas_per_sm(norm_bwd_kernel<K>, threads, fit[p.C / 16], (size_t)depth * row);
  const int64_t grid = std::min<int64_t>(
      std::min<int64_t>(p.R, (int64_t)sm_count() * per_sm), std::max<int64_t>(1, kNormPart / p.C));
  e = launch_pdl_smem(norm_bwd_kernel<K>, dim3((unsigned)grid), dim3(threads),
                      (size_t)depth * row, st, p, depth);
  if (e != cudaSuccess) return e;
  return launch_pdl(column_sum_kernel, dim3((unsigned)((p.C + 31) / 32)), dim3(kSumWarps * 32), st,
                    (const float*)p.part, (int)grid, (int)p.C, p.gw);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int target, bool fos, cudaStream_t st) {
  if (target == 0) return sized<kMx, false>(p, st);
  if (p.gamax) return fos ? sized<kTensor, true>(p, st) : sized<kTensor, false>(p, st);
  return fos ? sized<kRow, true>(p, st) : sized<kRow, false>(p, st);
}

cudaError_t launch_norm_bwd(const NormBwdParams& p, cudaStream_t st) {
  const int chunks = p.C / 8;
  if (chunks <= kMaxThreads) return run_bwd<1>(p, st);
  if (chunks <= 2 * kMaxThreads) return run_bwd<2>(p, st);
  return run_bwd<4>(p, st);
}

}  // namespace nvfp4
