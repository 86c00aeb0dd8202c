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
// (forward) and 6 (backward) bytes per value. Measured at 40 heads of 128, normed:
// forward 8192 tokens 29.3 us (5.87 TB/s, 87% of the measured copy rate), 32 tokens 2.0
// us; gradient 8192 tokens 53.8 us (4.76 TB/s, 70%), 65536 tokens 366 us (83%). The two
// lie 5.4 ns per token apart, 85% of the copy rate, and leave about 10 us of a call that do
// not depend on the tokens: its start, and the weights' gradients over warps, CTAs and
// then in the last CTA.
#include "kv.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;      // forward
constexpr int kWarps = kThreads / 32;
// Gradient: one CTA per SM (half the rows of sums to add up at the end), with 128
// registers a thread for four heads in flight (8192 tokens: 54.5 us; two in flight 62;
// 384 threads 63; 640, 768 and 1024 spill: 59 to 82).
constexpr int kThreadsBwd = 512;
constexpr int kWarpsBwd = kThreadsBwd / 32;
constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kBatch = 4;  // steps whose loads are in flight together

// A lane's 8 values as the two members of its four pairs, two pairs to an f32x2
// (one instruction works on two values): pair i is (a[i / 2], b[i / 2]) in the same
// half of both. The memory words w0 .. w3 hold values 0 1, 2 3, .. (of the lane's
// first and second group): with halves, w0 w1 are the first members and w2 w3 their
// partners; interleaved, a word is a pair.
struct V8 {
  f2 a[2], b[2];
};
template <bool IL>
__device__ __forceinline__ V8 unpack(const uint2& u, const uint2& w) {
  V8 x;
  if constexpr (IL) {
    x.a[0] = make_float2(bf16_lo(u.x), bf16_lo(u.y)), x.b[0] = make_float2(bf16_hi(u.x), bf16_hi(u.y));
    x.a[1] = make_float2(bf16_lo(w.x), bf16_lo(w.y)), x.b[1] = make_float2(bf16_hi(w.x), bf16_hi(w.y));
  } else {
    x.a[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x)), x.a[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
    x.b[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x)), x.b[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
  }
  return x;
}
// Value j (0 .. 7 in memory order) of the lane.
template <bool IL>
__device__ __forceinline__ float value(const V8& x, int j) {
  const f2 v = IL ? (j & 1 ? x.b[j >> 2] : x.a[j >> 2]) : (j < 4 ? x.a[j >> 1] : x.b[(j - 4) >> 1]);
  return (IL ? (j >> 1) & 1 : j & 1) ? v.y : v.x;
}
__device__ __forceinline__ V8 mul(const V8& x, const V8& y) {
  return {{f2_mul(x.a[0], y.a[0]), f2_mul(x.a[1], y.a[1])},
          {f2_mul(x.b[0], y.b[0]), f2_mul(x.b[1], y.b[1])}};
}
__device__ __forceinline__ V8 scale(const V8& x, float f) {
  const f2 ff = make_float2(f, f);
  return {{f2_mul(x.a[0], ff), f2_mul(x.a[1], ff)}, {f2_mul(x.b[0], ff), f2_mul(x.b[1], ff)}};
}
// x y + z
__device__ __forceinline__ V8 fma(const V8& x, const V8& y, const V8& z) {
  return {{f2_fma(x.a[0], y.a[0], z.a[0]), f2_fma(x.a[1], y.a[1], z.a[1])},
          {f2_fma(x.b[0], y.b[0], z.b[0]), f2_fma(x.b[1], y.b[1], z.b[1])}};
}
// x f + z
__device__ __forceinline__ V8 fma(const V8& x, float f, const V8& z) {
  const f2 ff = make_float2(f, f);
  return {{f2_fma(x.a[0], ff, z.a[0]), f2_fma(x.a[1], ff, z.a[1])},
          {f2_fma(x.b[0], ff, z.b[0]), f2_fma(x.b[1], ff, z.b[1])}};
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
struct Angles {
  f2 c[2], s[2];
  template <class L>
  __device__ __forceinline__ void load(const L& ln, const float* cs, int R) {
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
    if (ln.on) {
      a = *reinterpret_cast<const float4*>(cs + ln.angle);
      b = *reinterpret_cast<const float4*>(cs + R / 2 + ln.angle);
    }
    c[0] = make_float2(a.x, a.y), c[1] = make_float2(a.z, a.w);
    s[0] = make_float2(b.x, b.y), s[1] = make_float2(b.z, b.w);
  }
  // (a, b) -> (a c - b s, b c + a s), by the opposite angle if BACK.
  template <bool BACK>
  __device__ __forceinline__ void rotate(V8& x, bool on) const {
    if (!on) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f2 n = make_float2(-s[i].x, -s[i].y), a = x.a[i], b = x.b[i];
      x.a[i] = f2_fma(b, BACK ? s[i] : n, f2_mul(a, c[i]));
      x.b[i] = f2_fma(a, BACK ? n : s[i], f2_mul(b, c[i]));
    }
  }
};

// Every sum over the lanes of its head.
template <int LPH, int N>
__device__ __forceinline__ void head_sums(float (&v)[N]) {
#pragma unroll
  for (int d = LPH / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(kAll, v[i], d));
}
__device__ __forceinline__ float dot8(const V8& x, const V8& y) {
  f2 e = f2_mul(x.a[0], y.a[0]);
  e = f2_fma(x.a[1], y.a[1], e);
  e = f2_fma(x.b[0], y.b[0], e);
  e = f2_fma(x.b[1], y.b[1], e);
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
template <bool IL, class L>
__device__ __forceinline__ void store8(uint16_t* head, const L& ln, const V8& x) {
  *reinterpret_cast<uint2*>(head + ln.d0) =
      make_uint2(pack_bf16x2(value<IL>(x, 0), value<IL>(x, 1)),
                 pack_bf16x2(value<IL>(x, 2), value<IL>(x, 3)));
  *reinterpret_cast<uint2*>(head + ln.d1) =
      make_uint2(pack_bf16x2(value<IL>(x, 4), value<IL>(x, 5)),
                 pack_bf16x2(value<IL>(x, 6), value<IL>(x, 7)));
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

// A launch's warp tasks: `per` consecutive steps (heads of one tensor and token).
// The queries' tasks come first, then the keys': a task never mixes the two, so its
// weight and addresses are the warp's.
struct Tasks {
  int steps[2], tasks[2], per;  // of q and of k
  FastDiv by_tasks[2];
  int64_t total_q, total;
};
struct Task {
  bool k;
  int64_t t;
  int s0, s1;
};
__device__ __forceinline__ Task task_of(const Tasks& g, int64_t w) {
  Task x;
  x.k = w >= g.total_q;
  const int64_t u = x.k ? w - g.total_q : w;
  const int n = x.k ? g.tasks[1] : g.tasks[0];
  x.t = g.total < 0xFFFFFFFFll ? (int64_t)fastdiv((uint32_t)u, x.k ? g.by_tasks[1] : g.by_tasks[0])
                               : u / n;
  x.s0 = (int)(u - x.t * n) * g.per;
  x.s1 = min(x.s0 + g.per, x.k ? g.steps[1] : g.steps[0]);
  return x;
}

// The first loads go out before the token's position (whose angles depend on it) is
// waited for. Weight and angles are multiplied once per task: with x r the normed
// pair, a' = r (x_a (c w_a) - x_b (s w_b)) and b' = r (x_b (c w_b) + x_a (s w_a)).
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreads, 4) qk_rope_kernel(const QkRopeParams p, const Tasks g) {
  pdl_begin();
  using L = Lane<LPH, IL>;
  constexpr int D = 8 * LPH;
  const L ln(p.R);
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= g.total) return;
  const Task k = task_of(g, w);
  const int H = k.k ? p.hk : p.hq;
  const uint4* weight = k.k ? p.kw : p.qw;
  const uint16_t* in = (k.k ? p.k + k.t * p.k_st : p.q + k.t * p.q_st) + ln.sub * D;
  uint16_t* out = (k.k ? p.ko + k.t * p.ko_st : p.qo + k.t * p.qo_st) + ln.sub * D;
  V8 c, n;  // what a member is multiplied by for itself and for its partner
  for (int s = k.s0; s < k.s1; s += kBatch) {
    Raw raw[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      raw[b] = {make_uint2(0, 0), make_uint2(0, 0)};
      if (s + b < k.s1 && (s + b) * L::kHeads + ln.sub < H)
        raw[b] = load8(in + (s + b) * (L::kHeads * D), ln);
    }
    if (s == k.s0) {
      const Raw rw = weight8(weight, ln);
      Angles an;
      an.load(ln, p.cs + position(p, k.t) * p.R, p.R);
      const V8 wt = unpack<IL>(rw.a, rw.b);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c.a[i] = f2_mul(wt.a[i], an.c[i]);
        c.b[i] = f2_mul(wt.b[i], an.c[i]);
        n.a[i] = f2_mul(wt.a[i], an.s[i]);
        n.b[i] = f2_mul(wt.b[i], make_float2(-an.s[i].x, -an.s[i].y));
      }
      if (!ln.on) c = wt;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (s + b >= k.s1) break;
      V8 x = unpack<IL>(raw[b].a, raw[b].b);
      if (weight) {
        float ss[1] = {dot8(x, x)};
        head_sums<LPH>(ss);
        x = scale(x, rsqrtf(__fmaf_rn(ss[0], 1.0f / D, p.eps)));
      }
      V8 y = mul(x, c);
      if (ln.on) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          y.a[i] = f2_fma(x.b[i], n.b[i], y.a[i]);
          y.b[i] = f2_fma(x.a[i], n.a[i], y.b[i]);
        }
      }
      if ((s + b) * L::kHeads + ln.sub < H) store8<IL>(out + (s + b) * (L::kHeads * D), ln, y);
    }
  }
}

// Gradient: persistent warps over the tasks; each lane keeps the weight gradients of
// its 8 values, of the queries and, once its tasks are the keys', of the keys. A
// CTA's sums go to its row of the workspace, and the CTA that takes the last ticket
// adds the rows in order: the sums do not depend on which CTA finishes when.
template <int LPH, bool IL>
__global__ void __launch_bounds__(kThreadsBwd, 1) qk_rope_bwd_kernel(const QkRopeParams p,
                                                                  const Tasks g) {
  pdl_begin();
  using L = Lane<LPH, IL>;
  constexpr int D = 8 * LPH;
  const L ln(p.R);
  const int warp = threadIdx.x >> 5;
  V8 sum = {}, sum_q = {};
  bool keys = false;
  for (int64_t w = (int64_t)blockIdx.x * kWarpsBwd + warp; w < g.total;
       w += (int64_t)gridDim.x * kWarpsBwd) {
    const Task k = task_of(g, w);
    if (k.k && !keys) {
      keys = true;
      sum_q = sum;
      sum = {};
    }
    const int H = k.k ? p.hk : p.hq;
    const uint4* weight = k.k ? p.kw : p.qw;
    const uint16_t* gin = (k.k ? p.gk + k.t * p.gk_st : p.gq + k.t * p.gq_st) + ln.sub * D;
    const uint16_t* in = (k.k ? p.k + k.t * p.k_st : p.q + k.t * p.q_st) + ln.sub * D;
    uint16_t* out = (k.k ? p.ko + k.t * p.ko_st : p.qo + k.t * p.qo_st) + ln.sub * D;
    Angles an;
    V8 wt;
    for (int s = k.s0; s < k.s1; s += kBatch) {
      Raw rg[kBatch], rx[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        rg[b] = rx[b] = {make_uint2(0, 0), make_uint2(0, 0)};
        if (s + b < k.s1 && (s + b) * L::kHeads + ln.sub < H) {
          rg[b] = load8(gin + (s + b) * (L::kHeads * D), ln);
          if (weight) rx[b] = load8(in + (s + b) * (L::kHeads * D), ln);
        }
      }
      if (s == k.s0) {
        const Raw rw = weight8(weight, ln);
        an.load(ln, p.cs + position(p, k.t) * p.R, p.R);
        wt = unpack<IL>(rw.a, rw.b);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (s + b >= k.s1) break;
        const bool ok = (s + b) * L::kHeads + ln.sub < H;
        V8 u = unpack<IL>(rg[b].a, rg[b].b);
        an.rotate<true>(u, ln.on);
        if (weight) {
          const V8 x = unpack<IL>(rx[b].a, rx[b].b), wu = mul(u, wt);
          float v[2] = {dot8(x, x), dot8(wu, x)};
          head_sums<LPH>(v);
          const float r = rsqrtf(__fmaf_rn(v[0], 1.0f / D, p.eps));
          const V8 xr = scale(x, r);
          if (ok) sum = fma(u, xr, sum);  // (a head that is not there may have r infinite)
          // r (w u - x r^2 mean(w u x)) = r w u - (x r) (r mean) r: r^2 may be past fp32
          u = fma(xr, -__fmul_rn(__fmul_rn(__fmul_rn(v[1], 1.0f / D), r), r), scale(wu, r));
        }
        if (ok) store8<IL>(out + (s + b) * (L::kHeads * D), ln, u);
      }
    }
  }
  const V8 aq = keys ? sum_q : sum, ak = keys ? sum : V8{};
  if (!p.gqw && !p.gkw) return;

  // the CTA's sums: over the heads side by side in a warp, then over warps
  __shared__ float s_sum[kWarpsBwd][2 * D];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float vq = value<IL>(aq, j), vk = value<IL>(ak, j);
#pragma unroll
    for (int d = LPH; d < 32; d <<= 1) {
      vq = __fadd_rn(vq, __shfl_xor_sync(kAll, vq, d));
      vk = __fadd_rn(vk, __shfl_xor_sync(kAll, vk, d));
    }
    if (ln.sub == 0) {
      const int at = j < 4 ? ln.d0 + j : ln.d1 + j - 4;
      s_sum[warp][at] = vq;
      s_sum[warp][D + at] = vk;
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kThreadsBwd) {
    float v = s_sum[0][c];
#pragma unroll
    for (int i = 1; i < kWarpsBwd; ++i) v = __fadd_rn(v, s_sum[i][c]);
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
  // four adjacent columns per thread, the rows dealt to the groups of threads
  constexpr int kCols4 = 2 * D / 4, kGroups = kThreadsBwd / kCols4;
  const int c4 = threadIdx.x % kCols4, grp = threadIdx.x / kCols4;
  float4 a = make_float4(0, 0, 0, 0);
  const float4* rows = reinterpret_cast<const float4*>(p.ws);
#pragma unroll 16
  for (int i = grp; i < gridDim.x; i += kGroups) {
    const float4 v = __ldcg(rows + (int64_t)i * kCols4 + c4);
    a.x = __fadd_rn(a.x, v.x), a.y = __fadd_rn(a.y, v.y);
    a.z = __fadd_rn(a.z, v.z), a.w = __fadd_rn(a.w, v.w);
  }
  float4* s4 = reinterpret_cast<float4*>(&s_sum[0][0]);  // kGroups x kCols4 <= kWarpsBwd x 2 D floats
  static_assert(kGroups * kCols4 * 4 <= kWarpsBwd * 2 * D, "sums fit");
  s4[grp * kCols4 + c4] = a;
  __syncthreads();
  const float* s1 = &s_sum[0][0];
  for (int c = threadIdx.x; c < 2 * D; c += kThreadsBwd) {
    float v = s1[c];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) v = __fadd_rn(v, s1[i * 2 * D + c]);
    float* dst = c < D ? p.gqw : p.gkw;
    if (dst) dst[c < D ? c : c - D] = v;
  }
  if (threadIdx.x == 0) *ticket = 0;
}

// Steps per warp task: as many as still fill the GPU with warps, `most` at most (the
// gradient's persistent warps share the tasks out: fewer steps, smaller remainders).
Tasks make_tasks(const QkRopeParams& p, int heads, int most) {
  Tasks g{};
  g.steps[0] = (p.hq + heads - 1) / heads;
  g.steps[1] = (p.hk + heads - 1) / heads;
  const int64_t warps = (int64_t)sm_count() * 64;
  auto count = [&](int per) {
    return (g.steps[0] + per - 1) / per + (g.steps[1] + per - 1) / per;
  };
  int per = std::max(g.steps[0], g.steps[1]);
  while (per > 1 && p.T * count(per) < warps) per = (per + 1) / 2;
  g.per = std::min(per, most);
  for (int i = 0; i < 2; ++i) {
    g.tasks[i] = (g.steps[i] + g.per - 1) / g.per;
    g.by_tasks[i] = make_fastdiv((uint32_t)std::max(g.tasks[i], 1));
  }
  g.total_q = p.T * g.tasks[0];
  g.total = g.total_q + p.T * g.tasks[1];
  return g;
}

template <int LPH, bool IL>
cudaError_t fwd(const QkRopeParams& p, cudaStream_t st) {
  const Tasks g = make_tasks(p, 32 / LPH, 4 * kBatch);
  const int64_t ctas = (g.total + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(qk_rope_kernel<LPH, IL>, dim3((unsigned)ctas), dim3(kThreads), st, p, g);
}
template <int LPH, bool IL>
cudaError_t bwd(const QkRopeParams& p, cudaStream_t st) {
  const Tasks g = make_tasks(p, 32 / LPH, 2 * kBatch);
  static const int per_sm = resident_ctas(qk_rope_bwd_kernel<LPH, IL>, kThreadsBwd);
  const int64_t cap = std::min<int64_t>((int64_t)sm_count() * per_sm, kQkMaxCtas);
  const int64_t ctas = std::min<int64_t>((g.total + kWarpsBwd - 1) / kWarpsBwd, cap);
  return launch_pdl(qk_rope_bwd_kernel<LPH, IL>, dim3((unsigned)ctas), dim3(kThreadsBwd), st, p, g);
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
