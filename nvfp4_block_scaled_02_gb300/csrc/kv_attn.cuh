// kv_attn.cuh -- device building blocks shared by the two attention kernels
// over the NVFP4 cache: conversions, the exponential, and a request's key range.
#pragma once
#include "kv.h"

namespace nvfp4 {

constexpr unsigned kAll = 0xFFFFFFFFu;
// Probabilities enter the second product times 2^kBias (f16 keeps 11 bits down
// to 2^-14), and a running maximum may lag kSlack powers of two behind.
constexpr int kBias = 6;
constexpr float kSlack = 8.0f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 scale bytes (low 16 bits) -> f16x2, exact.
__device__ __forceinline__ uint32_t scales2(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
      : "=r"(r) : "r"(b));
  return r;
}
// 8 codes of a word -> 4 f16x2 (byte i: low nibble in the low half).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A request's rows and keys. rows = query tokens; keys [lo, hi) are seen by
// some row, lo rounded down to a tile.
struct Request {
  int q0, n, len, lo16, tiles;
};
__device__ __forceinline__ Request request(const KvAttnParams& p, int b, bool& bad) {
  Request r;
  r.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  r.len = p.seq_len[b];
  r.n = q1 - r.q0;
  bad = r.q0 < 0 || q1 < r.q0 || q1 > p.T || r.n > p.max_q || r.len < 0 ||
        r.len > INT32_MAX - 1024 || (int64_t)r.len > (int64_t)p.cols * p.P;
  if (bad) r.q0 = r.n = r.len = 0;
  int lo = 0;
  if (p.window > 0) lo = max(0, r.len - r.n + 1 - min(p.window, r.len));
  r.lo16 = lo & ~15;
  r.tiles = r.n > 0 ? (r.len - r.lo16 + 15) >> 4 : 0;
  return r;
}

}  // namespace nvfp4
