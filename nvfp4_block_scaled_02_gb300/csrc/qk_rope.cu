// qk_rope.cu -- RMS norm of every query and key head and the rotation of its
// position in one pass, and the gradient of both.
//
// Forward, per head x of D values: y = x r w with r = rsqrt(mean(x^2) + eps),
// then (a, b) -> (a c - b s, b c + a s) for every rotated pair of y.
// Backward: u = the output's gradient rotated by the opposite angle; gw = sum
// over rows of u x r; gx = r (w u - x r^2 mean(w u x)).
//
// A head lies in D/8 adjacent lanes (8 values, one 128-bit load each): the
// mean is a butterfly over those lanes, and a pair (i, i + R/2) is exchanged
// by one shuffle per value (R/16 lanes away). A warp takes several heads of
// one token in a row, so that the token's cosines and sines stay in registers.
// Both directions are bound by DRAM: 4 (forward) and 6 (backward) bytes per
// value, with some 3 instructions per value between.
#include "kv.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kBatch = 4;  // steps whose loads are in flight together

struct V8 {
  float v[8];
};
__device__ __forceinline__ V8 unpack(const uint4& w) {
  return {{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), bf16_lo(w.z), bf16_hi(w.z),
           bf16_lo(w.w), bf16_hi(w.w)}};
}
__device__ __forceinline__ uint4 pack(const V8& x) {
  return make_uint4(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]),
                    pack_bf16x2(x.v[4], x.v[5]), pack_bf16x2(x.v[6], x.v[7]));
}

// The cosines and sines of one lane's 8 values. Halves layout: value i and its
// partner share angle i mod R/2; the sine is negated in the first half, so
// that y = x c + partner s in both (and, with s negated, the inverse).
// Interleaved: angle k of the pair (2k, 2k + 1) in c[k], s[k], k < 4.
// A lane past the rotated part passes its values through (on = false).
template <bool IL>
struct Angles {
  float c[IL ? 4 : 8] = {}, s[IL ? 4 : 8] = {};
  bool on;
  __device__ __forceinline__ void load(const float* cs, int R, int d0) {
    constexpr int N = IL ? 4 : 8;
    on = d0 < R;
    if (on) {
      const bool first = d0 < R / 2;
      const int i = IL ? d0 / 2 : (first ? d0 : d0 - R / 2);
#pragma unroll
      for (int j = 0; j < N; j += 4) {
        const float4 a = *reinterpret_cast<const float4*>(cs + i + j);
        const float4 b = *reinterpret_cast<const float4*>(cs + R / 2 + i + j);
        c[j] = a.x, c[j + 1] = a.y, c[j + 2] = a.z, c[j + 3] = a.w;
        s[j] = b.x, s[j + 1] = b.y, s[j + 2] = b.z, s[j + 3] = b.w;
      }
      if (!IL && first)
#pragma unroll
        for (int j = 0; j < N; ++j) s[j] = -s[j];
    }
  }
  __device__ __forceinline__ void negate() {
#pragma unroll
    for (int j = 0; j < (IL ? 4 : 8); ++j) s[j] = -s[j];
  }
  // Rotates the lane's values; `partner` is the lane holding the other members
  // (halves layout). Every lane of the warp calls this.
  __device__ __forceinline__ V8 rotate(const V8& x, int partner) const {
    V8 y;
    if constexpr (IL) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = x.v[2 * k], b = x.v[2 * k + 1];
        y.v[2 * k] = __fmaf_rn(-b, s[k], __fmul_rn(a, c[k]));
        y.v[2 * k + 1] = __fmaf_rn(a, s[k], __fmul_rn(b, c[k]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o = __shfl_sync(kAll, x.v[j], partner);
        y.v[j] = __fmaf_rn(o, s[j], __fmul_rn(x.v[j], c[j]));
      }
    }
    return on ? y : x;
  }
};

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float dot8(const V8& a, const V8& b) {
  float e = 0.0f, o = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    e = __fmaf_rn(a.v[j], b.v[j], e);
    o = __fmaf_rn(a.v[j + 1], b.v[j + 1], o);
  }
  return __fadd_rn(e, o);
}

// What a lane does for its head in every step of a warp.
template <int LPH>
struct Lane {
  static constexpr int kHeads = 32 / LPH;  // heads per step
  int sub, l, d0, partner;
  __device__ explicit Lane(int R) {
    const int lane = threadIdx.x & 31;
    sub = lane / LPH;
    l = lane % LPH;
    d0 = 8 * l;
    const int far = R / 16;
    partner = d0 >= R ? lane : d0 < R / 2 ? lane + far : lane - far;
  }
};

__device__ __forceinline__ int64_t position(const QkRopeParams& p, int64_t t) {
  const int64_t pos = p.pos[t];
  if (pos >= 0 && pos < p.max_pos) return pos;
  flag(p.status, kDevBadIndex);
  return 0;
}

// Warp task: `per` consecutive steps of one token.
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const QkRopeParams p, int steps,
                                                           int per, FastDiv by_tasks, int tasks) {
  pdl_begin();
  using L = Lane<LPH>;
  const L ln(p.R);
  const int H = p.hq + p.hk;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.T * tasks) return;
  const int64_t t = w < 0xFFFFFFFFll ? (int64_t)fastdiv((uint32_t)w, by_tasks) : w / tasks;
  const int s0 = (int)(w - t * tasks) * per, s1 = min(s0 + per, steps);
  Angles<IL> an;
  an.load(p.cs + position(p, t) * p.R, p.R, ln.d0);
  const V8 one = {{1, 1, 1, 1, 1, 1, 1, 1}};
  const V8 wq = p.qw ? unpack(p.qw[ln.l]) : one, wk = p.kw ? unpack(p.kw[ln.l]) : one;
  const int64_t q_in = t * p.q_st + ln.d0, k_in = t * p.k_st + ln.d0;
  const int64_t q_out = t * p.qo_st + ln.d0, k_out = t * p.ko_st + ln.d0;
  for (int s = s0; s < s1; s += kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = (s + b) * L::kHeads + ln.sub;
      raw[b] = make_uint4(0, 0, 0, 0);
      if (s + b < s1 && h < H)
        raw[b] = *reinterpret_cast<const uint4*>(
            h < p.hq ? p.q + q_in + h * (8 * LPH) : p.k + k_in + (h - p.hq) * (8 * LPH));
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (s + b >= s1) break;
      const int h = (s + b) * L::kHeads + ln.sub;
      const bool is_q = h < p.hq;
      V8 x = unpack(raw[b]);
      const float ss = head_sum<LPH>(dot8(x, x));
      if (is_q ? p.qw != nullptr : p.kw != nullptr) {
        const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / (8 * LPH)), p.eps));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x.v[j] = __fmul_rn(__fmul_rn(x.v[j], r), is_q ? wq.v[j] : wk.v[j]);
      }
      const V8 y = an.rotate(x, ln.partner);
      if (h < H)
        *reinterpret_cast<uint4*>(is_q ? p.qo + q_out + h * (8 * LPH)
                                       : p.ko + k_out + (h - p.hq) * (8 * LPH)) = pack(y);
    }
  }
}

// Gradient: persistent warps over (token, chunk of steps); each lane keeps the
// weight gradients of its 8 values. A CTA's sums go to its row of the
// workspace, and the CTA that takes the last ticket adds the rows in order:
// the sums do not depend on which CTA finishes when.
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreads) qk_rope_bwd_kernel(const QkRopeParams p, int steps,
                                                               int per, FastDiv by_tasks,
                                                               int tasks) {
  pdl_begin();
  using L = Lane<LPH>;
  constexpr int D = 8 * LPH;
  const L ln(p.R);
  const int H = p.hq + p.hk;
  const int warp = threadIdx.x >> 5;
  const V8 one = {{1, 1, 1, 1, 1, 1, 1, 1}};
  const V8 wq = p.qw ? unpack(p.qw[ln.l]) : one, wk = p.kw ? unpack(p.kw[ln.l]) : one;
  V8 aq = {}, ak = {};
  const int64_t total = p.T * tasks;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < total;
       w += (int64_t)gridDim.x * kWarps) {
    const int64_t t = total < 0xFFFFFFFFll ? (int64_t)fastdiv((uint32_t)w, by_tasks) : w / tasks;
    const int s0 = (int)(w - t * tasks) * per, s1 = min(s0 + per, steps);
    Angles<IL> an;
    an.load(p.cs + position(p, t) * p.R, p.R, ln.d0);
    an.negate();
    for (int s = s0; s < s1; s += kBatch) {
      uint4 rg[kBatch], rx[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = (s + b) * L::kHeads + ln.sub;
        const bool ok = s + b < s1 && h < H, is_q = h < p.hq;
        const int64_t at = (is_q ? h : h - p.hq) * D + ln.d0;
        rg[b] = rx[b] = make_uint4(0, 0, 0, 0);
        if (ok) {
          rg[b] = *reinterpret_cast<const uint4*>((is_q ? p.gq + t * p.gq_st : p.gk + t * p.gk_st) + at);
          if (is_q ? p.qw != nullptr : p.kw != nullptr)
            rx[b] = *reinterpret_cast<const uint4*>((is_q ? p.q + t * p.q_st : p.k + t * p.k_st) + at);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (s + b >= s1) break;
        const int h = (s + b) * L::kHeads + ln.sub;
        const bool is_q = h < p.hq;
        const V8 x = unpack(rx[b]);
        V8 u = an.rotate(unpack(rg[b]), ln.partner);
        const float ss = head_sum<LPH>(dot8(x, x));
        const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps));
        V8 wu;
#pragma unroll
        for (int j = 0; j < 8; ++j) wu.v[j] = __fmul_rn(u.v[j], is_q ? wq.v[j] : wk.v[j]);
        const float m = head_sum<LPH>(dot8(wu, x));
        if (h < H && (is_q ? p.qw != nullptr : p.kw != nullptr)) {
          const float f = __fmul_rn(__fmul_rn(r, r), __fmul_rn(m, 1.0f / D));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float e = __fmul_rn(u.v[j], __fmul_rn(x.v[j], r));
            if (is_q) aq.v[j] = __fadd_rn(aq.v[j], e);
            else ak.v[j] = __fadd_rn(ak.v[j], e);
            u.v[j] = __fmul_rn(r, __fmaf_rn(-x.v[j], f, wu.v[j]));
          }
        }
        if (h < H) {
          const int64_t at = (is_q ? h : h - p.hq) * D + ln.d0;
          *reinterpret_cast<uint4*>((is_q ? p.qo + t * p.qo_st : p.ko + t * p.ko_st) + at) = pack(u);
        }
      }
    }
  }
  if (!p.gqw && !p.gkw) return;

  // the CTA's sums: over the heads side by side in a warp, then over warps
  __shared__ float s_sum[kWarps][2 * D];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int d = LPH; d < 32; d <<= 1) {
      aq.v[j] = __fadd_rn(aq.v[j], __shfl_xor_sync(kAll, aq.v[j], d));
      ak.v[j] = __fadd_rn(ak.v[j], __shfl_xor_sync(kAll, ak.v[j], d));
    }
    if (ln.sub == 0) {
      s_sum[warp][ln.d0 + j] = aq.v[j];
      s_sum[warp][D + ln.d0 + j] = ak.v[j];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    float v = s_sum[0][c];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) v = __fadd_rn(v, s_sum[i][c]);
    p.ws[(int64_t)blockIdx.x * 2 * D + c] = v;
  }
  uint32_t* ticket = reinterpret_cast<uint32_t*>(p.ws + (size_t)kQkMaxCtas * 2 * 128);
  __shared__ bool s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(ticket, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // four adjacent columns per thread, the rows dealt to kThreads / (D/2) groups
  constexpr int kCols4 = 2 * D / 4, kGroups = kThreads / kCols4;
  const int c4 = threadIdx.x % kCols4, grp = threadIdx.x / kCols4;
  float4 a = make_float4(0, 0, 0, 0);
  const float4* rows = reinterpret_cast<const float4*>(p.ws);
#pragma unroll 8
  for (int i = grp; i < gridDim.x; i += kGroups) {
    const float4 v = __ldcg(rows + (int64_t)i * kCols4 + c4);
    a.x = __fadd_rn(a.x, v.x), a.y = __fadd_rn(a.y, v.y);
    a.z = __fadd_rn(a.z, v.z), a.w = __fadd_rn(a.w, v.w);
  }
  float4* s4 = reinterpret_cast<float4*>(&s_sum[0][0]);  // kGroups x kCols4 <= kWarps x 2 D floats
  static_assert(kGroups * kCols4 * 4 <= kWarps * 2 * D, "sums fit");
  s4[grp * kCols4 + c4] = a;
  __syncthreads();
  const float* s1 = &s_sum[0][0];
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    float v = s1[c];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) v = __fadd_rn(v, s1[i * 2 * D + c]);
    float* dst = c < D ? p.gqw : p.gkw;
    if (dst) dst[c < D ? c : c - D] = v;
  }
  if (threadIdx.x == 0) *ticket = 0;
}

// Steps per warp task: as many as still fill the GPU with warps, 8 at most.
int steps_per_task(int64_t T, int steps) {
  const int64_t warps = (int64_t)sm_count() * 64;
  int per = steps;
  while (per > 1 && T * ((steps + per - 1) / per) < warps) per = (per + 1) / 2;
  return std::min(per, 8);
}

template <int LPH, bool IL>
cudaError_t fwd(const QkRopeParams& p, cudaStream_t st) {
  const int steps = (p.hq + p.hk + 32 / LPH - 1) / (32 / LPH);
  const int per = steps_per_task(p.T, steps), tasks = (steps + per - 1) / per;
  const int64_t ctas = (p.T * tasks + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(qk_rope_kernel<LPH, IL>, dim3((unsigned)ctas), dim3(kThreads), st, p, steps,
                    per, make_fastdiv((uint32_t)tasks), tasks);
}
template <int LPH, bool IL>
cudaError_t bwd(const QkRopeParams& p, cudaStream_t st) {
  const int steps = (p.hq + p.hk + 32 / LPH - 1) / (32 / LPH);
  const int per = steps_per_task(p.T, steps), tasks = (steps + per - 1) / per;
  static const int per_sm = resident_ctas(qk_rope_bwd_kernel<LPH, IL>, kThreads);
  const int64_t cap = std::min<int64_t>((int64_t)sm_count() * per_sm, kQkMaxCtas);
  const int64_t ctas = std::min<int64_t>((p.T * tasks + kWarps - 1) / kWarps, cap);
  return launch_pdl(qk_rope_bwd_kernel<LPH, IL>, dim3((unsigned)ctas), dim3(kThreads), st, p,
                    steps, per, make_fastdiv((uint32_t)tasks), tasks);
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeParams& p, int D, bool il, cudaStream_t st) {
  if (D == 128) return il ? fwd<16, true>(p, st) : fwd<16, false>(p, st);
  return il ? fwd<8, true>(p, st) : fwd<8, false>(p, st);
}
cudaError_t launch_qk_rope_bwd(const QkRopeParams& p, int D, bool il, cudaStream_t st) {
  if (D == 128) return il ? bwd<16, true>(p, st) : bwd<16, false>(p, st);
  return il ? bwd<8, true>(p, st) : bwd<8, false>(p, st);
}

}  // namespace nvfp4
