// qk_rope.cu -- RMS norm of every query and key head and the rotation of its
// position in one pass, and the gradient of both.
//
// Forward, per head x of D values: y = x r w with r = rsqrt(mean(x^2) + eps),
// then (a, b) -> (a c - b s, b c + a s) for every rotated pair of y.
// Backward: u = the output's gradient rotated by the opposite angle; gw = sum
// over rows of u x r; gx = r (w u - x r^2 mean(w u x)).
//
// A head lies in D/8 adjacent lanes, 8 values each: the mean is a butterfly over
// those lanes. With rotated halves a lane holds values 4l .. 4l + 3 and their
// partners R/2 on (two 64-bit loads), with interleaved pairs 8 values in a row:
// either way a pair never leaves its lane, four angles serve eight values, and the
// rotation needs no shuffle. A warp takes several heads of one token in a row, so
// that the token's angles stay in registers. Both directions are bound by DRAM: 4
// (forward) and 6 (backward) bytes per value.
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
__device__ __forceinline__ V8 unpack(const uint2& a, const uint2& b) {
  return {{bf16_lo(a.x), bf16_hi(a.x), bf16_lo(a.y), bf16_hi(a.y), bf16_lo(b.x), bf16_hi(b.x),
           bf16_lo(b.y), bf16_hi(b.y)}};
}

// Where a lane's two groups of four values lie in its head, and its angles.
template <int LPH, bool IL>
struct Lane {
  static constexpr int kHeads = 32 / LPH;  // heads per warp step
  int sub, d0, d1;
  bool on;      // the lane's values are rotated
  int angle;    // of its first pair
  __device__ explicit Lane(int R) {
    const int lane = threadIdx.x & 31, l = lane % LPH;
    sub = lane / LPH;
    on = 8 * l < R;
    d0 = !IL && on ? 4 * l : 8 * l;
    d1 = !IL && on ? 4 * l + R / 2 : 8 * l + 4;
    angle = 4 * l;
  }
};
template <bool IL>
struct Angles {
  float4 c, s;
  template <int LPH>
  __device__ __forceinline__ void load(const Lane<LPH, IL>& ln, const float* cs, int R) {
    c = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (ln.on) {
      c = *reinterpret_cast<const float4*>(cs + ln.angle);
      s = *reinterpret_cast<const float4*>(cs + R / 2 + ln.angle);
    }
  }
  __device__ __forceinline__ void negate() { s = make_float4(-s.x, -s.y, -s.z, -s.w); }
  static __device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float x = a;
    a = __fmaf_rn(-b, s, __fmul_rn(x, c));
    b = __fmaf_rn(x, s, __fmul_rn(b, c));
  }
  // Pairs (j, j + 4) of the lane, or (2j, 2j + 1). Values that are not rotated pass
  // through: 1 x + 0 y is x unless y is infinite, so they are left alone.
  __device__ __forceinline__ void rotate(V8& x, bool on) const {
    if (!on) return;
    if constexpr (IL) {
      turn(x.v[0], x.v[1], c.x, s.x);
      turn(x.v[2], x.v[3], c.y, s.y);
      turn(x.v[4], x.v[5], c.z, s.z);
      turn(x.v[6], x.v[7], c.w, s.w);
    } else {
      turn(x.v[0], x.v[4], c.x, s.x);
      turn(x.v[1], x.v[5], c.y, s.y);
      turn(x.v[2], x.v[6], c.z, s.z);
      turn(x.v[3], x.v[7], c.w, s.w);
    }
  }
};

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float dot8(const V8& a, const V8& b) {
  f2 e = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    e = f2_fma(make_float2(a.v[j], a.v[j + 1]), make_float2(b.v[j], b.v[j + 1]), e);
  return __fadd_rn(e.x, e.y);
}

// The values of one lane of a head as they are in memory.
struct Raw {
  uint2 a, b;
};
template <class L>
__device__ __forceinline__ Raw load8(const uint16_t* head, const L& ln) {
  return {*reinterpret_cast<const uint2*>(head + ln.d0),
          *reinterpret_cast<const uint2*>(head + ln.d1)};
}
template <class L>
__device__ __forceinline__ void store8(uint16_t* head, const L& ln, const V8& x) {
  *reinterpret_cast<uint2*>(head + ln.d0) =
      make_uint2(pack_bf16x2(x.v[0], x.v[1]), pack_bf16x2(x.v[2], x.v[3]));
  *reinterpret_cast<uint2*>(head + ln.d1) =
      make_uint2(pack_bf16x2(x.v[4], x.v[5]), pack_bf16x2(x.v[6], x.v[7]));
}
// A weight's values for this lane, or ones.
template <class L>
__device__ __forceinline__ Raw weight8(const uint4* w, const L& ln) {
  if (!w) return {make_uint2(0x3F803F80u, 0x3F803F80u), make_uint2(0x3F803F80u, 0x3F803F80u)};
  return load8(reinterpret_cast<const uint16_t*>(w), ln);
}

__device__ __forceinline__ int64_t position(const QkRopeParams& p, int64_t t) {
  const int64_t pos = p.pos[t];
  if (pos >= 0 && pos < p.max_pos) return pos;
  flag(p.status, kDevBadIndex);
  return 0;
}

// Warp task: `per` consecutive steps of one token. The first loads go out before
// the token's position (whose angles depend on it) is waited for.
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const QkRopeParams p, int steps,
                                                           int per, FastDiv by_tasks, int tasks) {
  pdl_begin();
  using L = Lane<LPH, IL>;
  constexpr int D = 8 * LPH;
  const L ln(p.R);
  const int H = p.hq + p.hk;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= p.T * tasks) return;
  const int64_t t = w < 0xFFFFFFFFll ? (int64_t)fastdiv((uint32_t)w, by_tasks) : w / tasks;
  const int s0 = (int)(w - t * tasks) * per, s1 = min(s0 + per, steps);
  const uint16_t *q = p.q + t * p.q_st, *k = p.k + t * p.k_st - (int64_t)p.hq * D;
  uint16_t *qo = p.qo + t * p.qo_st, *ko = p.ko + t * p.ko_st - (int64_t)p.hq * D;
  Angles<IL> an;
  Raw wq, wk;
  for (int s = s0; s < s1; s += kBatch) {
    Raw raw[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = (s + b) * L::kHeads + ln.sub;
      raw[b] = {make_uint2(0, 0), make_uint2(0, 0)};
      if (s + b < s1 && h < H) raw[b] = load8((h < p.hq ? q : k) + h * D, ln);
    }
    if (s == s0) {
      wq = weight8(p.qw, ln);
      wk = weight8(p.kw, ln);
      an.load(ln, p.cs + position(p, t) * p.R, p.R);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (s + b >= s1) break;
      const int h = (s + b) * L::kHeads + ln.sub;
      const bool is_q = h < p.hq;
      V8 x = unpack(raw[b].a, raw[b].b);
      const float ss = head_sum<LPH>(dot8(x, x));
      if (is_q ? p.qw != nullptr : p.kw != nullptr) {
        const float r = rsqrtf(__fmaf_rn(ss, 1.0f / D, p.eps));
        const V8 wt = unpack(is_q ? wq.a : wk.a, is_q ? wq.b : wk.b);
#pragma unroll
        for (int j = 0; j < 8; ++j) x.v[j] = __fmul_rn(__fmul_rn(x.v[j], r), wt.v[j]);
      }
      an.rotate(x, ln.on);
      if (h < H) store8((is_q ? qo : ko) + h * D, ln, x);
    }
  }
}

// Gradient: persistent warps over (token, chunk of steps); each lane keeps the
// weight gradients of its 8 values. A CTA's sums go to its row of the
// workspace, and the CTA that takes the last ticket adds the rows in order:
// the sums do not depend on which CTA finishes when.
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreads, 2) qk_rope_bwd_kernel(const QkRopeParams p, int steps,
                                                                  int per, FastDiv by_tasks,
                                                                  int tasks) {
  pdl_begin();
  using L = Lane<LPH, IL>;
  constexpr int D = 8 * LPH;
  const L ln(p.R);
  const int H = p.hq + p.hk;
  const int warp = threadIdx.x >> 5;
  const Raw wq = weight8(p.qw, ln), wk = weight8(p.kw, ln);
  V8 aq = {}, ak = {};
  const int64_t total = p.T * tasks;
  for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < total;
       w += (int64_t)gridDim.x * kWarps) {
    const int64_t t = total < 0xFFFFFFFFll ? (int64_t)fastdiv((uint32_t)w, by_tasks) : w / tasks;
    const int s0 = (int)(w - t * tasks) * per, s1 = min(s0 + per, steps);
    const int64_t k0 = -(int64_t)p.hq * D;
    const uint16_t *gq = p.gq + t * p.gq_st, *gk = p.gk + t * p.gk_st + k0;
    const uint16_t *q = p.q + t * p.q_st, *k = p.k + t * p.k_st + k0;
    uint16_t *qo = p.qo + t * p.qo_st, *ko = p.ko + t * p.ko_st + k0;
    Angles<IL> an;
    for (int s = s0; s < s1; s += kBatch) {
      Raw rg[kBatch], rx[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = (s + b) * L::kHeads + ln.sub;
        const bool is_q = h < p.hq;
        rg[b] = rx[b] = {make_uint2(0, 0), make_uint2(0, 0)};
        if (s + b < s1 && h < H) {
          rg[b] = load8((is_q ? gq : gk) + h * D, ln);
          if (is_q ? p.qw != nullptr : p.kw != nullptr) rx[b] = load8((is_q ? q : k) + h * D, ln);
        }
      }
      if (s == s0) {
        an.load(ln, p.cs + position(p, t) * p.R, p.R);
        an.negate();
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (s + b >= s1) break;
        const int h = (s + b) * L::kHeads + ln.sub;
        const bool is_q = h < p.hq;
        const V8 x = unpack(rx[b].a, rx[b].b);
        V8 u = unpack(rg[b].a, rg[b].b);
        an.rotate(u, ln.on);
        const V8 wt = unpack(is_q ? wq.a : wk.a, is_q ? wq.b : wk.b);
        V8 wu;
#pragma unroll
        for (int j = 0; j < 8; ++j) wu.v[j] = __fmul_rn(u.v[j], wt.v[j]);
        const float ss = head_sum<LPH>(dot8(x, x)), m = head_sum<LPH>(dot8(wu, x));
        if (h < H && (is_q ? p.qw != nullptr : p.kw != nullptr)) {
          const float r = rsqrtf(__fmaf_rn(ss, 1.0f / D, p.eps));
          const float f = __fmul_rn(__fmul_rn(r, r), __fmul_rn(m, 1.0f / D));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xr = __fmul_rn(x.v[j], r);
            if (is_q) aq.v[j] = __fmaf_rn(u.v[j], xr, aq.v[j]);
            else ak.v[j] = __fmaf_rn(u.v[j], xr, ak.v[j]);
            u.v[j] = __fmul_rn(r, __fmaf_rn(-x.v[j], f, wu.v[j]));
          }
        }
        if (h < H) store8((is_q ? qo : ko) + h * D, ln, u);
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
      const int at = j < 4 ? ln.d0 + j : ln.d1 + j - 4;
      s_sum[warp][at] = aq.v[j];
      s_sum[warp][D + at] = ak.v[j];
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
#pragma unroll 16
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
