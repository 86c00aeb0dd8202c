// kv_attn.cu -- attention over a paged KV cache held in NVFP4, for few query
// rows per KV head (single tokens and a few drafted ones, grouped heads).
//
//   out = softmax(scale q K^T) V over the keys a row sees,
//   K = code_k * scale_k * g_k, V = code_v * scale_v * g_v.
//
// Numerics. code * block scale has at most 2 + 4 significant bits and lies in
// [2^-10, 2688], so it is exact in f16; g_k goes into the softmax scale and
// g_v into the final division. A query row is multiplied by a power of two
// that puts its largest element in [2^13, 2^14): its bf16 elements are then
// exact in f16 down to 2^-27 of that one, and off by at most 2^-38 of it below.
// Scores, maxima, sums and outputs are fp32. The probabilities are rounded to
// f16 for the second product (2^-11 relative; the sum that divides them is
// taken before rounding), times 2^kBias so that they stay normal down to
// 2^-20 of the largest.
//
// One pass over K and V with a running maximum per row. The maximum is only
// raised (and the accumulators rescaled) when a score exceeds it by more than
// kSlack powers of two: the result is the same, the rescaling is rare, and
// 2^(kBias + kSlack) is far from f16's largest value.
//
// Work split. A query row block (the rows of one request that share a KV head)
// and its tiles of 16 tokens form an item; all items' costs and tiles, one after the
// other, are cut into equal runs, one per CTA, whatever the requests' lengths.
// An item cut between CTAs leaves a record (out, maximum, sum) per CTA in the
// workspace, and the CTA that takes the item's last ticket joins the records
// in order. Inside a CTA the warps take tiles in turn and join at the item's
// end. (With a CTA per item a call would last as long as its longest item does in one
// CTA; cut evenly, 64 ragged requests run at the rate of 64 equal ones.)
//
// What bounds it: DRAM and the conversions together. A tile of 16 keys is 2304 bytes
// and about 280 warp instructions, many of them conversions and byte moves on the ALU
// pipe, which is nearly half busy (issue slots 59%) at 79% of the measured copy rate. Measured,
// one row per request, 8 KV heads, groups of 4, D = 128: 64 requests x 8192 tokens 109
// us (5.54 TB/s, 82% of that rate); 64 ragged ones, 672 MB in all, 121 us (82%); 256 x
// 500 tokens 45 us (50%: an item is 8 tiles per warp and each costs its set-up and join);
// 4 requests of 300 to 1100 tokens 9.8 us (latency).
//
// Tile layout (m16n8k16, K or V as the 16-row operand, query rows as the 8
// columns). Lane (g, t) = (lane / 4, lane % 4). Which token a K row index
// stands for and which dimension a k index stands for are free as long as both
// products agree, so they are chosen for wide loads: lane t holds dimensions
// [t D/4, (t+1) D/4) of K rows g and g + 8 (one 128-bit load each), and lane g
// holds dimensions [g D/8, (g+1) D/8) of V for the tokens 4 i + t, i < 4. The
// probabilities of K rows (g, g + 8) become the second product's operand by an
// 8x8 transpose between lanes. Two V bytes of neighbouring tokens are merged
// to (even nibbles) and (odd nibbles) before conversion, so that a converted
// pair holds one dimension of two tokens, as the operand wants.
#include <cmath>
#include <cstddef>

#include "kv_attn.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// What an item costs beside its tiles (set-up and joins), in tiles. Without it the CTAs
// whose runs hold the most short items end last (256 requests of 16 to 16384 tokens, log-
// uniform: 188 us with 0, 161 with 8, 140 with 16, 139 with 24; 200 of 300 with 16 of
// 8192: 68, 57, 56, 60), and short items are cut for nothing (4 requests of 300 to 1100:
// 13.5 us with 0, 10.5 with the others).
constexpr int kItemCost = 16;
constexpr int kStages = 4;  // tiles in flight per warp (cp.async groups)
// A request this kernel takes.
__device__ __forceinline__ Request few_rows(const KvAttnParams& p, int b, bool& bad) {
  Request r = request(p, b, bad);
  const int64_t rows = (int64_t)r.n * p.G;
  if (rows <= p.over_rows || rows > p.few_rows) r.n = r.tiles = 0;
  return r;
}

// A run is counted in units: kItemCost for an item, then one per tile.
__device__ __forceinline__ int units(const Request& r) {
  return r.tiles > 0 ? r.tiles + kItemCost : 0;
}

template <int D>
struct Stage {
  uint8_t k[16 * D / 2], v[16 * D / 2], ks[16 * D / 16], vs[16 * D / 16];
};

// 16 bytes from global to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Padded row of the joined outputs (floats), and where the four values at
// float4 index q of a row lie in it: the writing lanes (g, t) then hit all banks.
template <int D>
constexpr int kJoinRow = D + 4;
template <int D>
__device__ __forceinline__ int join_at(int q) {
  return D == 128 ? (q ^ ((q >> 2) & 1)) * 4 : q * 4;
}

template <int D, int NT>
struct Layout {
  static constexpr size_t kStage = sizeof(Stage<D>) * kStages * kWarps;
  static constexpr size_t kJoin = (size_t)kWarps * 8 * NT * kJoinRow<D> * 4;
  static constexpr size_t kBytes = kStage + kJoin;
};

// Tiles [t0, t1) of KV head h of request b.
struct Segment {
  Request r;
  int b, h, t0, t1;
};

// Record of CTA c's part of an item that begins in CTA c0.
__device__ __forceinline__ float* record(const KvAttnParams& p, int c, int c0) {
  return p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * kAttnRecord;
}
// A row's final result: values d .. d + 3 of row rr (token, head of the group).
template <int D>
__device__ __forceinline__ void finish(const KvAttnParams& p, int q0, int h, int rr, int d,
                                       float4 v, float mx, float sum, float vg) {
  const int tk = (int)fastdiv((uint32_t)rr, p.by_group), hh = rr - tk * p.G;
  const int64_t orow = (int64_t)(q0 + tk) * p.hq + h * p.G + hh;
  const float f = sum == 0.0f ? 0.0f : vg / sum;
  reinterpret_cast<uint2*>(p.out)[orow * (D / 4) + d / 4] =
      make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
  if (p.lse && d == 0)
    p.lse[orow] = sum == 0.0f ? __int_as_float(0xFF800000) : (mx - kBias + log2f(sum)) * kLn2;
}
// Joins the records of CTAs c0 .. c1 in order, 8 in flight. (16 would take 5 us off
// one request of 32768 tokens, but their registers cost the tile loop 4%, inlined
// or not.)
template <int D>
__device__ __noinline__ void join_records(const KvAttnParams& p, int q0, int h, int nrows, int c0,
                                          int c1, float vg) {
  constexpr int U = 8;
  for (int i = threadIdx.x; i < nrows * (D / 4); i += kThreads) {
    const int rr = i / (D / 4), q = i % (D / 4);
    float mx = __int_as_float(0xFF800000), sum = 0.0f;
    float4 v = make_float4(0, 0, 0, 0);
    for (int c = c0; c <= c1; c += U) {
      float mc[U], lc[U];
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float* rec = record(p, min(c + u, c1), c0);
        mc[u] = __ldcg(rec + kAttnRows * 128 + rr);
        lc[u] = __ldcg(rec + kAttnRows * 129 + rr);
        x[u] = __ldcg(reinterpret_cast<const float4*>(rec + rr * D + 4 * q));
        if (c + u > c1) mc[u] = __int_as_float(0xFF800000);
      }
      float mn = mx;
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, mc[u]);
      if (mn == __int_as_float(0xFF800000)) {  // sums of 0, or NaN where the scores are
#pragma unroll
        for (int u = 0; u < U; ++u) sum += lc[u];
        continue;
      }
      const float a = ex2(mx - mn);
      sum *= a;
      v.x *= a, v.y *= a, v.z *= a, v.w *= a;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float e = ex2(mc[u] - mn);  // 0 without a maximum: a NaN stays
        sum = __fmaf_rn(lc[u], e, sum);
        v.x = __fmaf_rn(x[u].x, e, v.x), v.y = __fmaf_rn(x[u].y, e, v.y);
        v.z = __fmaf_rn(x[u].z, e, v.z), v.w = __fmaf_rn(x[u].w, e, v.w);
      }
      mx = mn;
    }
    finish<D>(p, q0, h, rr, 4 * q, v, mx, sum, vg);
  }
}

// NaN into the outputs of the rows that see a key with a NaN scale in the block of V that
// this lane holds, among the keys of this warp's tiles of a segment. `dst`: row 2 t of the
// warp's outputs in shared memory. Rare, and kept out of the tile loop's registers: the
// cache is read again.
template <int D, int NT>
__device__ __noinline__ void put_nan(const KvAttnParams& p, float* dst, const Segment& s) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int block = g / (128 / D), nrows = s.r.n * p.G;
  uint32_t hit = 0;  // bit 2 nt + i: row 8 nt + 2 t + i
#pragma unroll 1
  for (int j = s.t0 + (threadIdx.x >> 5); j < s.t1; j += kWarps) {
    const int tok = s.r.lo16 + j * 16, pg = (int)fastdiv((uint32_t)tok, p.by_page);
    int64_t page = p.table[(int64_t)s.b * p.cols + pg];
    if (page < 0 || page >= p.pages) page = 0;
    const uint64_t row = (uint64_t)((page * p.hk + s.h) * p.P + (tok - pg * p.P));
#pragma unroll 1
    for (int key = tok; key < min(tok + 16, s.r.len); ++key) {
      if ((p.vs[(row + (key - tok)) * (D / 16) + block] & 0x7F) != 0x7F) continue;
#pragma unroll 1
      for (int c = 0; c < 2 * NT; ++c) {
        const int rr = (c >> 1) * 8 + 2 * t + (c & 1);
        const int lim = s.r.len - s.r.n + (int)fastdiv((uint32_t)rr, p.by_group) + 1;
        if (rr < nrows && key < lim && (p.window == 0 || key >= lim - min(p.window, s.r.len)))
          hit |= 1u << c;
      }
    }
  }
#pragma unroll 1
  for (int c = 0; c < 2 * NT; ++c)
    if (hit >> c & 1)
      for (int q = g * (D / 32); q < (g + 1) * (D / 32); ++q)
        *reinterpret_cast<float4*>(dst + ((c >> 1) * 8 + (c & 1)) * kJoinRow<D> + join_at<D>(q)) =
            make_float4(NAN, NAN, NAN, NAN);
}

// CTAs per SM that the compiler keeps registers for; as many run as then fit. For up
// to 8 rows at D = 128 a bound of three is best (145 registers): the loads and
// conversions of a tile overlap better than under a bound of four (64 requests x 8192
// tokens, 8 KV heads: 109 us, against 122 with four, and 113 to 117 held to 160 to 136
// registers). At D = 64 four: 75 us, against 76 with three and 85 with five. Up to 16
// rows: at D = 128 two (four rows a request: 153 us, against 163 with three, and 359
// with four, which spills), at D = 64 three (95 us, against 105 with two and 106 with
// four). Loading an item's queries under the one before it took registers from the tile
// loop and was no faster (64 x 8192: 112 us).
template <int D, int NT>
constexpr int kCtasPerSm = D == 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<D, NT>)
    kv_attn_kernel(const KvAttnParams p, const int ctas) {
  pdl_begin();
  constexpr int kRows = 8 * NT;  // query rows of an item at most
  constexpr int KS = D / 16;     // k steps of q K^T, and 16-row tiles of V^T
  constexpr int DQ = D / 4;      // dimensions of K per lane
  constexpr uint32_t kStageBytes = sizeof(Stage<D>);
  extern __shared__ __align__(16) uint8_t smem[];
  Stage<D>* stages = reinterpret_cast<Stage<D>*>(smem) + (threadIdx.x >> 5) * kStages;
  float* s_o = reinterpret_cast<float*>(smem + Layout<D, NT>::kStage);  // [kWarps][kRows][row]
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int s_b0;
  __shared__ int64_t s_off;
  __shared__ uint32_t s_ticket;
  __shared__ int s_nan[kWarps];  // a warp has left NaN blocks of V out of its products
  __shared__ Segment s_seg[kWarps];  // ... of this segment

  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(kAll, tid >> 5, 0);

  // ---- this CTA's run of tiles: a scan over the requests -------------------
  const int share = (p.B + kThreads - 1) / kThreads;
  const int rb0 = min(tid * share, p.B), rb1 = min(rb0 + share, p.B);
  int64_t mine = 0;
  for (int b = rb0; b < rb1; ++b) {
    bool bad;
    const Request r = few_rows(p, b, bad);
    if (bad && blockIdx.x == 0) flag(p.status, kDevBadIndex);
    mine += (int64_t)units(r) * p.hk;
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (lane == 0) s_nan[warp] = 0;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += s_scan[w];
    total += s_scan[w];
  }
  // equal runs, 8 units at least
  const int64_t run = max((total + ctas - 1) / ctas, (int64_t)(2 * kWarps));
  const int64_t first = (int64_t)blockIdx.x * run, last = min(first + run, total);
  if (first < last && incl - mine <= first && first < incl) {
    int64_t at = incl - mine;
    for (int b = rb0; b < rb1; ++b) {
      bool bad;
      const Request r = few_rows(p, b, bad);
      const int64_t c = (int64_t)units(r) * p.hk;
      if (first < at + c) {
        s_b0 = b;
        s_off = first - at;
        break;
      }
      at += c;
    }
  }

  // ---- rows that see no key ------------------------------------------------
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    bool bad;
    const Request r = few_rows(p, b, bad);
    if (r.n == 0 || r.tiles > 0) continue;
    const int64_t rows = (int64_t)r.n * p.hq;
    for (int64_t i = tid; i < rows * (D / 8); i += kThreads)
      reinterpret_cast<uint4*>(p.out)[(int64_t)r.q0 * p.hq * (D / 8) + i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t i = tid; i < rows; i += kThreads)
        p.lse[(int64_t)r.q0 * p.hq + i] = __int_as_float(0xFF800000);
  }
  __syncthreads();
  if (first >= last) return;

  // ---- segments: what this CTA does of each item it meets ------------------
  int64_t pos = first;  // tiles of the run not yet in a segment start here
  Segment seg;
  seg.b = s_b0;
  bool bad0;
  seg.r = few_rows(p, seg.b, bad0);
  seg.h = (int)(s_off / units(seg.r));
  auto take = [&](Segment& s, int from) -> bool {  // its tiles from unit `from` on; any?
    const int more = (int)min((int64_t)units(s.r) - from, last - pos);
    pos += more;
    s.t0 = max(from - kItemCost, 0);
    s.t1 = from + more - kItemCost;
    return s.t1 > s.t0;
  };
  auto next = [&](Segment& s) -> bool {  // the one after s, which it replaces
    if (pos >= last) return false;
    if (++s.h == p.hk) {
      s.h = 0;
      do {
        if (++s.b >= p.B) return false;
        bool bad;
        s.r = few_rows(p, s.b, bad);
      } while (s.r.tiles == 0);
    }
    return take(s, 0);
  };
  // (false: the run ends before its only item's tiles begin)
  if (!take(seg, (int)(s_off - (int64_t)seg.h * units(seg.r)))) return;
  // A segment's tile j is this warp's when j = t0 + warp mod 4. Lane l holds the
  // cache row of the first key of its l-th tile from `from` on: one table look-up
  // for 32 tiles, well before the copies that need it.
  auto look_up = [&](const Segment& s, int from) -> uint32_t {
    const int j = from + lane * kWarps;
    if (j >= s.t1) return 0;
    const int tok = s.r.lo16 + j * 16;
    int pg, of;
    if (p.page_shift >= 0) {
      pg = tok >> p.page_shift;
      of = tok & (p.P - 1);
    } else {
      pg = (int)fastdiv((uint32_t)tok, p.by_page);
      of = tok - pg * p.P;
    }
    int64_t page = p.table[(int64_t)s.b * p.cols + pg];
    if (page < 0 || page >= p.pages) {
      page = 0;
      flag(p.status, kDevBadIndex);
    }
    return (uint32_t)((page * p.hk + s.h) * p.P + of);
  };
  // Copies 16 keys from cache row `row` on into a stage: 16-byte chunks lane
  // and lane + 32 (D = 128) of the tile's K and V codes, one chunk of the scales.
  // What depends on the lane alone is worked out here, once.
  constexpr int CPR = D / 32;  // 16-byte chunks of a code row
  const int ctk = lane / CPR, cpart = lane % CPR;
  // K row index of the token (the inverse of token = 4 (r & 1) + r / 2 + 8 (r / 8))
  const int ckr = 2 * (ctk & 3) + ((ctk >> 2) & 1) + 8 * (ctk >> 3);
  // V chunks swapped so that lanes (g, t) read 4 tokens without bank conflicts
  const int cvp = D == 128 ? cpart ^ (((ctk >> 1) & 1) << 1) : cpart;
  const uint32_t stage0 = (uint32_t)__cvta_generic_to_shared(stages);
  const uint32_t k_dst = stage0 + ckr * (D / 2) + cpart * 16;
  const uint32_t v_dst = stage0 + offsetof(Stage<D>, v) + ctk * (D / 2) + cvp * 16;
  const uint32_t sc_dst = stage0 + offsetof(Stage<D>, ks) + lane * 16;  // ks, vs are neighbours
  const uint8_t* k_src = p.kc + lane * 16;
  const uint8_t* v_src = p.vc + lane * 16;
  const uint8_t* sc_src = lane < D / 16 ? p.ks + lane * 16 : p.vs + (lane - D / 16) * 16;
  auto copy = [&](uint32_t row, uint32_t at) {  // at: the stage's offset
    const uint8_t* ks = k_src + (uint64_t)row * (D / 2);
    const uint8_t* vs = v_src + (uint64_t)row * (D / 2);
    copy16(k_dst + at, ks);
    copy16(v_dst + at, vs);
    if constexpr (D == 128) {  // the tile's second 8 tokens: 8 rows on in both places
      copy16(k_dst + at + 512, ks + 512);
      copy16(v_dst + at + 512, vs + 512);
    }
    if (lane < D / 8) copy16(sc_dst + at, sc_src + (uint64_t)row * (D / 16));
  };
  // Where this lane reads a stage: K rows g and g + 8 with their scales, the V
  // bytes and scales of tokens t, 4 + t, 8 + t, 12 + t.
  const int tg = (g >> 1) + 4 * (g & 1);  // token of K row g; row g + 8: token tg + 8
  const uint32_t k_ld = stage0 + g * (D / 2) + t * (DQ / 2);
  const uint32_t ks_ld = stage0 + offsetof(Stage<D>, ks) + tg * (D / 16) + t * (D / 64);
  const uint32_t v_ld =
      stage0 + offsetof(Stage<D>, v) + t * (D / 2) +
      (D == 128 ? ((g >> 1) ^ (((t >> 1) & 1) << 1)) * 16 + (g & 1) * 8 : g * 4);
  const uint32_t vs_ld =
      stage0 + offsetof(Stage<D>, vs) + t * (D / 16) + (D == 128 ? g : g >> 1);
  // The first copies of a segment.
  auto begin = [&](const Segment& s, uint32_t rows) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const uint32_t row = __shfl_sync(kAll, rows, i);
      if (s.t0 + warp + i * kWarps < s.t1) copy(row, i * kStageBytes);
      cp_async_commit();
    }
  };

  // The query rows of a segment's item as they are in memory (column n of row tile
  // nt is row 8 nt + n = (token, head of the group)), and its heads' amax.
  uint4 raw[NT][DQ / 8];
  float k_amax = 0.0f, v_amax = 0.0f;
  auto load_q = [&](const Segment& s) {
    k_amax = p.k_amax[s.h];
    v_amax = p.v_amax[s.h];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g;
      const int tk = (int)fastdiv((uint32_t)row, p.by_group), hh = row - tk * p.G;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (s.r.q0 + tk) * p.q_st + (int64_t)(s.h * p.G + hh) * D + t * DQ);
#pragma unroll
      for (int i = 0; i < DQ / 8; ++i)
        raw[nt][i] = row < s.r.n * p.G ? src[i] : make_uint4(0, 0, 0, 0);
    }
  };

  uint32_t rows = look_up(seg, seg.t0 + warp);
  begin(seg, rows);
  bool have = true;
  while (have) {
    // the segment after this one: its rows are looked up now, its first copies run
    // while this one's results are joined
    const Request r = seg.r;
    const int h = seg.h, t0 = seg.t0, t1 = seg.t1;
    load_q(seg);
    const int64_t item_first = pos - t1, item_last = item_first + r.tiles - 1;  // its tiles' units
    const int nrows = r.n * p.G;
    if (lane == 0) s_seg[warp] = seg;
    __syncwarp();
    have = next(seg);
    uint32_t next_rows = have ? look_up(seg, seg.t0 + warp) : 0;

    // ---- query rows ---------------------------------------------------------
    uint32_t qb[NT][KS][2];
    float fac[NT][2];     // scores to powers of two, for columns 2t and 2t + 1
    int lim[NT][2];       // keys below this are seen
    const SliceScale kss = slice_scale(k_amax, p.M), vss = slice_scale(v_amax, p.M);
    if ((kss.bad || vss.bad) && tid == 0) flag(p.status, NVFP4_DEV_BAD_AMAX_BIT);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < DQ / 8; ++i) m = max(m, absmax_bits4(raw[nt][i]));
      m = max(m, __shfl_xor_sync(kAll, m, 1));
      m = max(m, __shfl_xor_sync(kAll, m, 2));
      if (m >= 0x7F80u) flag(p.status, NVFP4_DEV_NONFINITE_INPUT_BIT);
      // 2^(13 - e) for a row whose largest element lies in [2^e, 2^(e+1))
      const int e = min(max(13 - ((int)(m >> 7) - 127), -126), 126);
      float up = __uint_as_float((uint32_t)(127 + e) << 23);
      float f = p.scale * kLog2e * kss.g * __uint_as_float((uint32_t)(127 - e) << 23);
      if (f < 0.0f) f = -f, up = -up;  // maxima are taken before the factor: f > 0
      f = fmaxf(f, 1.17549435e-38f);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(raw[nt]);
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qb[nt][j][i] = pack_f16x2(bf16_lo(w[2 * j + i]) * up, bf16_hi(w[2 * j + i]) * up);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fac[nt][i] = __shfl_sync(kAll, f, (2 * t + i) * 4);
        const int rr = nt * 8 + 2 * t + i;
        lim[nt][i] = rr < nrows ? r.len - r.n + (int)fastdiv((uint32_t)rr, p.by_group) + 1 : 0;
      }
    }
    const int lim_min = r.len - r.n + 1;  // keys below are seen by every row
    const int low_max = p.window > 0 ? r.len - min(p.window, r.len) : 0;  // and from here on
    float o[NT][KS][4];
    float m[NT][2], l[NT][2];
    float sub[NT][2], above[NT][2];  // bias - m; the score above which m is raised
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[nt][i] = above[nt][i] = __int_as_float(0xFF800000);
        l[nt][i] = sub[nt][i] = 0.0f;
      }
    }

    // ---- tiles --------------------------------------------------------------
    uint32_t at = 0, fill = (kStages - 1) * kStageBytes;  // stages read and filled now
    int ahead = kStages - 1;                              // this warp's tiles copied so far
    uint32_t more_rows = look_up(s_seg[warp], t0 + warp + 32 * kWarps);  // its tiles 32 .. 63
    int tok = r.lo16 + (t0 + warp) * 16;
    const int tok_end = r.lo16 + t1 * 16, tok_fill = tok_end - (kStages - 1) * kWarps * 16;
    for (; tok < tok_end; tok += kWarps * 16) {
      const uint32_t row = __shfl_sync(kAll, rows, ahead & 31);
      if (tok < tok_fill) copy(row, fill);
      cp_async_commit();
      fill = at;  // the next one to fill is the one read now
      if ((++ahead & 31) == 0) {
        rows = more_rows;
        more_rows = look_up(s_seg[warp], t0 + warp + (ahead + 32) * kWarps);
      }
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const bool edge = tok + 16 > lim_min || tok < low_max;

      // scores: S^T[token][row]
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[nt][c] = 0.0f;
      {
        uint32_t ka[DQ / 8], kb[DQ / 8], sa, sb;
        if constexpr (D == 128) {
          const uint4 a = lds128(k_ld + at), b = lds128(k_ld + at + 8 * (D / 2));
          ka[0] = a.x, ka[1] = a.y, ka[DQ / 8 - 2] = a.z, ka[DQ / 8 - 1] = a.w;
          kb[0] = b.x, kb[1] = b.y, kb[DQ / 8 - 2] = b.z, kb[DQ / 8 - 1] = b.w;
          // block scales of the two rows as f16x2: two blocks
          sa = scales2(lds16(ks_ld + at));
          sb = scales2(lds16(ks_ld + at + 8 * (D / 16)));
        } else {
          const uint2 a = lds64(k_ld + at), b = lds64(k_ld + at + 8 * (D / 2));
          ka[0] = a.x, ka[1] = a.y, kb[0] = b.x, kb[1] = b.y;
          sa = scales2(lds8(ks_ld + at));
          sb = scales2(lds8(ks_ld + at + 8 * (D / 16)));
        }
#pragma unroll
        for (int i = 0; i < DQ / 8; ++i) {
          const uint32_t fa = __byte_perm(sa, 0, (D == 128 && i >= 2) ? 0x3232 : 0x1010);
          const uint32_t fb = __byte_perm(sb, 0, (D == 128 && i >= 2) ? 0x3232 : 0x1010);
          uint32_t ha[4], hb[4];
          codes8(ka[i], ha);
          codes8(kb[i], hb);
#pragma unroll
          for (int c = 0; c < 4; ++c) ha[c] = h2mul(ha[c], fa), hb[c] = h2mul(hb[c], fb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(sc[nt], ha[0], hb[0], ha[1], hb[1], qb[nt][2 * i][0], qb[nt][2 * i][1]);
            mma(sc[nt], ha[2], hb[2], ha[3], hb[3], qb[nt][2 * i + 1][0], qb[nt][2 * i + 1][1]);
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = tok + tg + 8 * (c >> 1), hi = lim[nt][c & 1];
            const bool seen = key < hi && (p.window == 0 || key >= hi - min(p.window, r.len));
            sc[nt][c] = seen ? sc[nt][c] : __int_as_float(0xFF800000);
          }
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) raise |= fmaxf(sc[nt][i], sc[nt][i + 2]) > above[nt][i];
      if (__any_sync(kAll, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(sc[nt][i], sc[nt][i + 2]);
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 4));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 8));
            x = fmaxf(x, __shfl_xor_sync(kAll, x, 16)) * fac[nt][i];
            const float mn = fmaxf(m[nt][i], x);
            // 0 for a row that has seen nothing yet (its sums are 0)
            const float a = m[nt][i] == __int_as_float(0xFF800000) ? 0.0f : ex2(m[nt][i] - mn);
            m[nt][i] = mn;
            if (mn != __int_as_float(0xFF800000)) {
              sub[nt][i] = kBias - mn;
              above[nt][i] = (mn + kSlack) / fac[nt][i];
            }
            l[nt][i] *= a;
#pragma unroll
            for (int d = 0; d < KS; ++d) o[nt][d][i] *= a, o[nt][d][i + 2] *= a;
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          e[c] = ex2(__fmaf_rn(sc[nt][c], fac[nt][c & 1], sub[nt][c & 1]));
        const f2 two = __fadd2_rn(make_float2(e[0], e[1]), make_float2(e[2], e[3]));
        l[nt][0] += two.x;
        l[nt][1] += two.y;
        pb[nt][0] = transpose8x8(pack_f16x2(e[0], e[1]));
        pb[nt][1] = transpose8x8(pack_f16x2(e[2], e[3]));
      }
      // K row 2t is token t, row 2t + 1 token 4 + t, rows + 8 tokens + 8
      {
        constexpr int VW = D / 64;  // words of a lane's V chunk
        uint32_t vw[4][VW], vb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint2 w = lds64(v_ld + at + 4 * i * (D / 2));
            vw[i][0] = w.x, vw[i][VW - 1] = w.y;
          } else {
            vw[i][0] = lds32(v_ld + at + 4 * i * (D / 2));
          }
          vb[i] = lds8(vs_ld + at + 4 * i * (D / 16));
        }
        // Bytes past the request may hold anything. And a NaN block of a key that some row
        // does not see would reach that row as 0 x NaN: it leaves the product, and the rows
        // that see it get the NaN at the end.
        if (edge) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (tok + 4 * i + t >= r.len) vb[i] = 0;
            if ((vb[i] & 0x7Fu) == 0x7Fu) vb[i] = 0, s_nan[warp] = 1;
          }
        }
        const uint32_t f01 = scales2(__byte_perm(vb[0], vb[1], 0x0040));
        const uint32_t f23 = scales2(__byte_perm(vb[2], vb[3], 0x0040));
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          const uint32_t e01 = (vw[0][w] & 0x0F0F0F0Fu) | ((vw[1][w] << 4) & 0xF0F0F0F0u);
          const uint32_t o01 = ((vw[0][w] >> 4) & 0x0F0F0F0Fu) | (vw[1][w] & 0xF0F0F0F0u);
          const uint32_t e23 = (vw[2][w] & 0x0F0F0F0Fu) | ((vw[3][w] << 4) & 0xF0F0F0F0u);
          const uint32_t o23 = ((vw[2][w] >> 4) & 0x0F0F0F0Fu) | (vw[3][w] & 0xF0F0F0F0u);
          uint32_t a0[4], a1[4], a2[4], a3[4];
          codes8(e01, a0);
          codes8(o01, a1);
          codes8(e23, a2);
          codes8(o23, a3);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            a0[c] = h2mul(a0[c], f01), a1[c] = h2mul(a1[c], f01);
            a2[c] = h2mul(a2[c], f23), a3[c] = h2mul(a3[c], f23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma(o[nt][4 * w + c], a0[c], a1[c], a2[c], a3[c], pb[nt][0], pb[nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the slot before it is filled again
      at = at == (kStages - 1) * kStageBytes ? 0 : at + kStageBytes;
    }
    cp_async_wait<0>();
    __syncwarp();
    rows = next_rows;
    if (have) begin(seg, rows);

    // ---- join the warps ------------------------------------------------------
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = l[nt][i];
        v += __shfl_xor_sync(kAll, v, 4);
        v += __shfl_xor_sync(kAll, v, 8);
        v += __shfl_xor_sync(kAll, v, 16);
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t + i] = m[nt][i];
          s_l[warp][nt * 8 + 2 * t + i] = v;
        }
        float* dst = s_o + (warp * kRows + nt * 8 + 2 * t + i) * kJoinRow<D>;
#pragma unroll
        for (int c = 0; c < KS; c += 2)
          *reinterpret_cast<float4*>(dst + join_at<D>(g * (D / 32) + c / 2)) =
              make_float4(o[nt][c][i], o[nt][c][i + 2], o[nt][c + 1][i], o[nt][c + 1][i + 2]);
      }
    if (s_nan[warp]) {
      put_nan<D, NT>(p, s_o + (warp * kRows + 2 * t) * kJoinRow<D>, s_seg[warp]);
      __syncwarp();
      if (lane == 0) s_nan[warp] = 0;
    }
    __syncthreads();
    const int c0 = (int)(item_first / run), c1 = (int)(item_last / run);  // CTAs of the item
    const bool whole = c0 == c1;
    for (int i = tid; i < nrows * (D / 4); i += kThreads) {
      const int rr = i / (D / 4), q = i % (D / 4);
      float mx = s_m[0][rr];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][rr]);
      float sum = 0.0f;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w][rr];
        const float a = mw == __int_as_float(0xFF800000) ? 0.0f : ex2(mw - mx);
        sum = __fmaf_rn(s_l[w][rr], a, sum);
        const float4 x =
            *reinterpret_cast<const float4*>(s_o + (w * kRows + rr) * kJoinRow<D> + join_at<D>(q));
        v.x = __fmaf_rn(x.x, a, v.x), v.y = __fmaf_rn(x.y, a, v.y);
        v.z = __fmaf_rn(x.z, a, v.z), v.w = __fmaf_rn(x.w, a, v.w);
      }
      if (whole) {
        finish<D>(p, r.q0, h, rr, 4 * q, v, mx, sum, vss.g);
      } else {
        float* rec = record(p, blockIdx.x, c0);
        *reinterpret_cast<float4*>(rec + rr * D + 4 * q) = v;
        if (q == 0) {
          rec[kAttnRows * 128 + rr] = mx;
          rec[kAttnRows * 129 + rr] = sum;
        }
      }
    }

    // ---- join the CTAs of a cut item ------------------------------------------
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) s_ticket = atomicAdd(p.tickets + c0, 1u);
      __syncthreads();
      if (s_ticket == (uint32_t)(c1 - c0)) {
        __threadfence();
        join_records<D>(p, r.q0, h, nrows, c0, c1, vss.g);
        if (tid == 0) p.tickets[c0] = 0;
      }
    }
    __syncthreads();  // the joined outputs have been read
  }
}

template <int D, int NT>
cudaError_t launch_t(const KvAttnParams& p, cudaStream_t st) {
  constexpr size_t smem = Layout<D, NT>::kBytes;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kv_attn_kernel<D, NT>, smem, ready);
  if (e != cudaSuccess) return e;
  static const int per_sm = resident_ctas(kv_attn_kernel<D, NT>, kThreads, smem);
  const int ctas = std::min(sm_count() * per_sm, kAttnMaxCtas);
  return launch_pdl_smem(kv_attn_kernel<D, NT>, dim3(ctas), dim3(kThreads), smem, st, p, ctas);
}

}  // namespace

// Requests of up to 8 rows and of 9 to 16 differ in the columns of their products (one
// row per request, 64 x 8192 tokens: 109 us with 8 columns, 152 with 16). Where a call
// may hold prompts besides (more than 16 rows), requests of both kinds are to be
// expected and each kind gets a launch (62 single rows at 8192 tokens with two prompts of
// 300: 143 us, against 188 in one; an empty launch adds 2 us to prompts alone); drafted
// tokens alone (16 rows at most) share the wider one.
cudaError_t launch_kv_few(KvAttnParams p, int D, cudaStream_t st) {
  const int64_t most = (int64_t)p.max_q * p.G;
  auto one = [&] { return D == 128 ? launch_t<128, 1>(p, st) : launch_t<64, 1>(p, st); };
  auto two = [&] { return D == 128 ? launch_t<128, 2>(p, st) : launch_t<64, 2>(p, st); };
  p.over_rows = 0;
  if (most <= 8) return one();
  if (most <= kAttnRows) return two();
  p.few_rows = 8;
  const cudaError_t e = one();
  if (e != cudaSuccess) return e;
  p.over_rows = 8;
  p.few_rows = kAttnRows;
  return two();
}

}  // namespace nvfp4
