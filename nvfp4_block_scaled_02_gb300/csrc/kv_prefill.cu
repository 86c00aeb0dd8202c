// kv_prefill.cu -- attention over a paged KV cache held in NVFP4, for many
// query rows per KV head (prompts): the two products on the tensor cores.
//
// The formula, the exactness of K and V in f16 and the numerics of the softmax
// are those of kv_attn.cu. Here a CTA takes 256 query rows of one KV head as
// two tiles of 128 (M), and walks over the keys in tiles of 128:
//   S = Q K^T  (Q, K in shared memory; S fp32 in tensor memory)
//   P = 2^(S f - m + bias), f16, written over S in tensor memory
//   O += P V   (P from tensor memory, V in shared memory; O fp32 in tensor memory)
// Tensor memory: S0 S1 (128 columns each), O0 O1 (D each): 512 columns at D = 128.
//
// Warps: 0-3 softmax of tile 0 (thread = row), 4-7 of tile 1, 8-11 dequantise K
// and V tiles into shared memory, 12 issues the MMAs, 13 hands out
// the items (14 and 15 only fill up their warpgroup, whose registers go to the
// softmax). While one tile's softmax
// runs, the other tile's products do. K and V tiles are double-buffered. All
// hand-overs are mbarriers; QK of the next tile is issued right behind PV of the
// previous one, so the barrier that says "S is ready" also says that the output
// accumulator may be rescaled.
//
// K and V are dequantised once per 256 query rows: 128 threads turn 16 bytes of
// codes into 32 f16 values each, in the 128-byte-swizzled layout the tensor
// cores read (K rows along k, V rows along n).
//
// Work split: as in kv_attn.cu, the items' key tiles are cut into equal runs, one
// per CTA; an item cut between CTAs is joined by the CTA that takes its last
// ticket, in order.
//
// Every wait has a limit: when it runs out the CTA sets NVFP4_DEV_TIMEOUT, its
// other waits return at once, and it frees its tensor memory and ends.
#include "kv_attn.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 512;  // 4 warpgroups
// Registers per thread: the softmax keeps a whole row of scores. Two softmax
// warpgroups, one that dequantises, one that issues: 2 x 184 + 80 + 64 = 4 x 128.
constexpr int kRegsSoftmax = 184, kRegsDequant = 80, kRegsMma = 64;
static_assert(2 * kRegsSoftmax + kRegsDequant + kRegsMma <= 4 * 128, "the block's registers");
constexpr int kTileN = 128;    // keys per tile
constexpr int kRowsTile = 128, kRowsItem = 256;
constexpr int kItems = 4;      // items handed out ahead
constexpr long long kWaitCycles = 2000000000;  // about a second
constexpr uint32_t kNegInf = 0xFF800000u;

struct Bars {
  uint64_t q_full[2], s_full[2], p_full[2], o_done[2];
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t item_full[kItems], item_free[kItems];
  uint64_t end;
};

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;  // bytes of a 128 x D f16 tile
  static constexpr size_t kBytes = 2 * kTile + 4 * (size_t)kTile + 1024;  // + alignment
};

// A request this kernel takes: more rows than the other kernel does.
__device__ __forceinline__ Request many_rows(const KvAttnParams& p, int b, bool& bad) {
  Request r = request(p, b, bad);
  if ((int64_t)r.n * p.G <= p.few_rows) r.n = 0;
  return r;
}
__device__ __forceinline__ int row_blocks(const KvAttnParams& p, const Request& r) {
  return r.len > 0 ? (r.n * p.G + kRowsItem - 1) / kRowsItem : 0;
}
// Key tiles of row block pt: [begin, begin + count), from its first row's lower
// limit to its last row's upper one. Rows that see nothing take one tile, too:
// they are written with it.
struct Tiles {
  int begin, count;
};
__device__ __forceinline__ Tiles block_tiles(const KvAttnParams& p, const Request& r, int pt) {
  const int last = min((pt + 1) * kRowsItem, r.n * p.G) - 1;
  const int hi = r.len - r.n + last / p.G + 1;
  int begin = 0;
  if (p.window > 0) {
    const int low = r.len - r.n + pt * kRowsItem / p.G + 1 - min(p.window, r.len);
    begin = max(0, low - r.lo16) / kTileN;
  }
  return {begin, max(1, (hi - r.lo16 + kTileN - 1) / kTileN - begin)};
}
__device__ __forceinline__ int64_t request_tiles(const KvAttnParams& p, const Request& r) {
  int64_t c = 0;
  const int n = row_blocks(p, r);
  for (int pt = 0; pt < n; ++pt) c += block_tiles(p, r, pt).count;
  return c * p.hk;
}

struct Item {
  Request r;
  int b, h, row0, rows;
  int t0, t1;     // this CTA's tiles, counted from key lo16
  int64_t first;  // the item's first tile in the run of all tiles
  int nt;         // all its tiles
};

// The items of this CTA's run [pos, last) of tiles, in the same order in every
// warp: row blocks inside heads inside requests.
struct Walk {
  int64_t pos, last;
  int64_t skip;  // tiles before pos, counted from (b, h, pt)
  int b, h, pt, blocks;
  Request r;
  __device__ void start(const KvAttnParams& p, int64_t first, int64_t end, int b0, int64_t off) {
    pos = first;
    last = end;
    b = b0;
    bool bad;
    r = many_rows(p, b, bad);
    blocks = row_blocks(p, r);
    const int64_t per_head = request_tiles(p, r) / p.hk;
    h = (int)(off / per_head);
    skip = off - h * per_head;
    pt = 0;
  }
  __device__ bool next(const KvAttnParams& p, Item& it) {
    while (pos < last) {
      if (pt == blocks) {
        pt = 0;
        if (++h == p.hk || blocks == 0) {
          h = 0;
          if (++b >= p.B) return false;
          bool bad;
          r = many_rows(p, b, bad);
          blocks = row_blocks(p, r);
        }
        continue;
      }
      const Tiles t = block_tiles(p, r, pt);
      if (skip >= t.count) {
        skip -= t.count;
        ++pt;
        continue;
      }
      const int count = (int)min((int64_t)t.count - skip, last - pos);
      it.r = r;
      it.b = b;
      it.h = h;
      it.row0 = pt * kRowsItem;
      it.rows = min(kRowsItem, r.n * p.G - it.row0);
      it.t0 = t.begin + (int)skip;
      it.t1 = it.t0 + count;
      it.first = pos - skip;
      it.nt = t.count;
      pos += count;
      skip += count;
      return true;
    }
    return false;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const KvAttnParams p,
                                                                 const int ctas) {
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bar;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_dead;
  __shared__ int64_t s_scan[kThreads / 32];
  __shared__ int s_b0;
  __shared__ int64_t s_off;
  __shared__ Item s_item[kItems];
  constexpr int kTile = Smem<D>::kTile;
  uint8_t* base = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* sq = base;               // [2] Q tiles
  uint8_t* sk = base + 2 * kTile;   // [2] K tiles
  uint8_t* sv = base + 4 * kTile;   // [2] V tiles

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- this CTA's run -------------------------------------------------------
  const int share = (p.B + kThreads - 1) / kThreads;
  const int rb0 = min(tid * share, p.B), rb1 = min(rb0 + share, p.B);
  int64_t mine = 0;
  for (int b = rb0; b < rb1; ++b) {
    bool bad;
    const Request r = many_rows(p, b, bad);
    if (bad && blockIdx.x == 0) flag(p.status, kDevBadIndex);
    mine += request_tiles(p, r);
  }
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid == 0) {
    s_dead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 128);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 128);
      mbar_init(&bar.o_done[i], 1);
      mbar_init(&bar.k_full[i], 128);
      mbar_init(&bar.v_full[i], 128);
      mbar_init(&bar.k_free[i], 1);
      mbar_init(&bar.v_free[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_free[i], 13);  // the softmax, dequantising and issuing warps
    }
    mbar_init(&bar.end, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) incl += s_scan[w];
    total += s_scan[w];
  }
  const int64_t run = max((total + ctas - 1) / ctas, (int64_t)2);
  const int64_t first = (int64_t)blockIdx.x * run, last = min(first + run, total);
  if (first < last && incl - mine <= first && first < incl) {
    int64_t at = incl - mine;
    for (int b = rb0; b < rb1; ++b) {
      bool bad;
      const int64_t c = request_tiles(p, many_rows(p, b, bad));
      if (first < at + c) {
        s_b0 = b;
        s_off = first - at;
        break;
      }
      at += c;
    }
  }

  // ---- requests without keys -------------------------------------------------
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    bool bad;
    const Request r = many_rows(p, b, bad);
    if (r.n == 0 || r.len > 0) continue;
    const int64_t rows = (int64_t)r.n * p.hq;
    for (int64_t i = tid; i < rows * (D / 8); i += kThreads)
      reinterpret_cast<uint4*>(p.out)[(int64_t)r.q0 * p.hq * (D / 8) + i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int64_t i = tid; i < rows; i += kThreads)
        p.lse[(int64_t)r.q0 * p.hq + i] = __uint_as_float(kNegInf);
  }
  if (first >= last) return;
  if (warp == 12) tmem_alloc(&s_tmem, 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  auto t_s = [&](int tile) { return tmem + 128 * tile; };
  auto t_o = [&](int tile) { return tmem + 256 + D * tile; };

  // A wait with a limit (kWaitCycles); false once the CTA gave up.
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    if (mbar_try(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(b, parity)) {
      if (s_dead) return false;
      if (clock64() - t0 > kWaitCycles) {
        s_dead = 1;
        flag(p.status, kDevTimeout);
        return false;
      }
    }
    return true;
  };
  // the same for a whole warp, whose lanes go on together
  auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(kAll, wait(b, parity));
  };

  // The item a warp is at: handed out by warp 13, one after the other, by way of
  // a ring; t1 = 0 ends the run.
  uint32_t items = 0;
  auto next = [&](const Item*& it) -> bool {
    if (items > 0) {
      __syncwarp();  // every lane is done with the last item
      if (lane == 0) mbar_arrive(&bar.item_free[(items - 1) % kItems]);
    }
    if (!wait_warp(&bar.item_full[items % kItems], (items / kItems) & 1)) return false;
    it = &s_item[items % kItems];
    ++items;
    return it->t1 > 0;
  };
  const Item* it;

  if (warp < 8) {
    // ==== softmax: thread = row of its tile ====================================
    more_registers<kRegsSoftmax>();
    const int tile = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane offset in a TMEM address
    const uint32_t ts = t_s(tile) + lanes, to = t_o(tile) + lanes;
    uint32_t sphase = 0, ophase = 0;
    bool ok = true;
    while (ok && next(it)) {
      if (tile * kRowsTile >= it->rows) continue;
      const Request r = it->r;
      const int rr = it->row0 + tile * kRowsTile + row;  // row of the request
      const bool live = rr < r.n * p.G;
      const int tk = live ? rr / p.G : 0, hh = rr - tk * p.G;
      const SliceScale kss = slice_scale(p.k_amax[it->h], p.M);
      const SliceScale vss = slice_scale(p.v_amax[it->h], p.M);
      if ((kss.bad || vss.bad) && row == 0) flag(p.status, NVFP4_DEV_BAD_AMAX_BIT);

      // -- query row: scaled to f16, into the swizzled tile
      float f;
      {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (int64_t)(r.q0 + tk) * p.q_st + (int64_t)(it->h * p.G + hh) * D);
        uint4 raw[D / 8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = live ? src[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) m = max(m, absmax_bits4(raw[i]));
        if (m >= 0x7F80u) flag(p.status, NVFP4_DEV_NONFINITE_INPUT_BIT);
        const int e = min(max(13 - ((int)(m >> 7) - 127), -126), 126);
        float up = __uint_as_float((uint32_t)(127 + e) << 23);
        f = p.scale * kLog2e * kss.g * __uint_as_float((uint32_t)(127 - e) << 23);
        if (f < 0.0f) f = -f, up = -up;  // the running maximum needs f > 0, and a masked
        f = fmaxf(f, 1.17549435e-38f);   // score (-inf) must stay -inf times f
        uint8_t* dst = sq + tile * kTile + row * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 w = raw[i];
          const uint4 h = make_uint4(pack_f16x2(bf16_lo(w.x) * up, bf16_hi(w.x) * up),
                                     pack_f16x2(bf16_lo(w.y) * up, bf16_hi(w.y) * up),
                                     pack_f16x2(bf16_lo(w.z) * up, bf16_hi(w.z) * up),
                                     pack_f16x2(bf16_lo(w.w) * up, bf16_hi(w.w) * up));
          *reinterpret_cast<uint4*>(dst + (i >> 3) * (128 * 128) + (((i & 7) ^ (row & 7)) << 4)) = h;
        }
      }
      fence_smem_async();
      mbar_arrive(&bar.q_full[tile]);

      // the row sees keys [low, low + span)
      const int lim = live ? r.len - r.n + tk + 1 : 0;
      const int low = p.window > 0 ? lim - min(p.window, r.len) : 0;
      const uint32_t span = (uint32_t)max(lim - low, 0);
      // keys in [safe_lo, safe_hi) are seen by every live row of the tile
      const int trow0 = it->row0 + tile * kRowsTile;
      const int trow1 = min(trow0 + kRowsTile, r.n * p.G) - 1;
      const int safe_hi = r.len - r.n + trow0 / p.G + 1;
      const int safe_lo = p.window > 0 ? r.len - r.n + trow1 / p.G + 1 - min(p.window, r.len) : 0;
      float m = __uint_as_float(kNegInf), l = 0.0f;

      const int t0 = it->t0, t1 = it->t1;
      for (int j = t0; j < t1; ++j) {
        if (!(ok = wait_warp(&bar.s_full[tile], sphase))) break;
        sphase ^= 1;
        fence_after();
        const int key0 = r.lo16 + j * kTileN;
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s[c]);
        tmem_wait_ld();
        if (key0 + kTileN > safe_hi || key0 < safe_lo) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((uint32_t)(key0 - low + 32 * c + i) >= span) s[c][i] = kNegInf;
        }
        float mx = __uint_as_float(kNegInf), mb = mx;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            mx = fmax3(mx, __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
            mb = fmax3(mb, __uint_as_float(s[c][i + 2]), __uint_as_float(s[c][i + 3]));
          }
        mx = fmaxf(mx, mb) * f;
        if (__any_sync(kAll, mx > m + kSlack)) {
          const float mn = fmaxf(m, mx);
          const float a = m == __uint_as_float(kNegInf) ? 0.0f : ex2(m - mn);
          m = mn;
          l *= a;
          if (j > t0) {  // S is ready, so PV of the previous tile is done
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(to + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
              tmem_st16(to + 16 * c, o);
            }
          }
        }
        const float sub = m == __uint_as_float(kNegInf) ? 0.0f : kBias - m;
        const f2 ff = make_float2(f, f), cc = make_float2(sub, sub);
        f2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f2 x = f2_fma(make_float2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])),
                          ff, cc);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum = __fadd2_rn(sum, x);
            h[i] = pack_f16x2(x.x, x.y);
          }
          tmem_st16(ts + 16 * c, h);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        fence_before();
        mbar_arrive(&bar.p_full[tile]);
      }
      if (!ok) break;

      // -- result: the whole row, or a record of this CTA's part of it
      if (!(ok = wait_warp(&bar.o_done[tile], ophase))) break;
      ophase ^= 1;
      fence_after();
      const int64_t c0 = it->first / run, c1 = (it->first + it->nt - 1) / run;
      uint32_t s[32];
      if (c0 == c1) {
        const float fo = l == 0.0f ? 0.0f : vss.g / l;
        const int64_t orow = (int64_t)(r.q0 + tk) * p.hq + it->h * p.G + hh;
        uint4* dst = reinterpret_cast<uint4*>(p.out) + orow * (D / 8);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          tmem_ld32(to + 32 * c, s);
          tmem_wait_ld();
          if (live)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* x = reinterpret_cast<const float*>(s) + 8 * i;
              dst[4 * c + i] = make_uint4(
                  pack_bf16x2(x[0] * fo, x[1] * fo), pack_bf16x2(x[2] * fo, x[3] * fo),
                  pack_bf16x2(x[4] * fo, x[5] * fo), pack_bf16x2(x[6] * fo, x[7] * fo));
            }
        }
        if (live && p.lse)
          p.lse[orow] =
              l == 0.0f ? __uint_as_float(kNegInf) : (m - kBias + log2f(l)) * kLn2;
      } else {
        // [D / 4][256 rows][4], then maxima and sums
        float* rec = p.part + ((int64_t)blockIdx.x * 2 + (blockIdx.x == c0 ? 1 : 0)) * kPrefillRecord;
        const int ri = tile * kRowsTile + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          tmem_ld32(to + 32 * c, s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            reinterpret_cast<uint4*>(rec)[(8 * c + i) * kRowsItem + ri] =
                make_uint4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
        }
        rec[kRowsItem * 128 + ri] = m;
        rec[kRowsItem * 129 + ri] = l;
        // a row is written by the same warp of every CTA: a ticket per warp
        __threadfence();
        __syncwarp();
        uint32_t* ticket = p.tickets + kAttnMaxCtas + 8 * c0 + warp;
        uint32_t mine_ticket = 0;
        if (lane == 0) mine_ticket = atomicAdd(ticket, 1u);
        if (__shfl_sync(kAll, mine_ticket, 0) == (uint32_t)(c1 - c0)) {
          __threadfence();
          float mx = __uint_as_float(kNegInf);
          for (int64_t c = c0; c <= c1; ++c)
            mx = fmaxf(mx, __ldcg(p.part + (c * 2 + (c == c0 ? 1 : 0)) * kPrefillRecord +
                                  kRowsItem * 128 + ri));
          float sum = 0.0f;
          for (int64_t c = c0; c <= c1; ++c) {
            const float* q = p.part + (c * 2 + (c == c0 ? 1 : 0)) * kPrefillRecord;
            const float mc = __ldcg(q + kRowsItem * 128 + ri);
            if (mc != __uint_as_float(kNegInf))
              sum += __ldcg(q + kRowsItem * 129 + ri) * ex2(mc - mx);
          }
          const float fo = sum == 0.0f ? 0.0f : vss.g / sum;
          const int64_t orow = (int64_t)(r.q0 + tk) * p.hq + it->h * p.G + hh;
          uint2* dst = reinterpret_cast<uint2*>(p.out) + orow * (D / 4);
#pragma unroll 4
          for (int d = 0; d < D / 4; ++d) {
            float4 v = make_float4(0, 0, 0, 0);
            for (int64_t c = c0; c <= c1; ++c) {
              const float* q = p.part + (c * 2 + (c == c0 ? 1 : 0)) * kPrefillRecord;
              const float mc = __ldcg(q + kRowsItem * 128 + ri);
              const float4 x = __ldcg(reinterpret_cast<const float4*>(q) + d * kRowsItem + ri);
              if (mc == __uint_as_float(kNegInf)) continue;
              const float w = ex2(mc - mx);
              v.x += x.x * w, v.y += x.y * w, v.z += x.z * w, v.w += x.w * w;
            }
            if (live)
              dst[d] = make_uint2(pack_bf16x2(v.x * fo, v.y * fo), pack_bf16x2(v.z * fo, v.w * fo));
          }
          if (live && p.lse)
            p.lse[orow] =
                sum == 0.0f ? __uint_as_float(kNegInf) : (mx - kBias + log2f(sum)) * kLn2;
          if (lane == 0) *ticket = 0;
        }
      }
    }
  } else if (warp < 12) {
    // ==== dequantise ============================================================
    fewer_registers<kRegsDequant>();
    // thread: rows 8 w + (lane & 7) + 32 i of a tile, 16-byte chunk lane / 8 of the
    // codes (D = 64: two row halves instead of four chunks)
    constexpr int kRowsPer = D == 128 ? 4 : 2;
    const int w = warp - 8;
    const int rbase = D == 128 ? w * 8 + (lane & 7) : w * 16 + (lane & 15);
    const int chunk = D == 128 ? lane >> 3 : lane >> 4;
    constexpr int kRowStep = D == 128 ? 32 : 64;
    uint32_t n = 0;  // tiles done
    bool ok = true;
    while (ok && next(it)) {
      const int32_t* table = p.table + (int64_t)it->b * p.cols;
      const int len = it->r.len;
      uint4 ck[kRowsPer], cv[kRowsPer];
      uint32_t bk[kRowsPer], bv[kRowsPer];
      int64_t at[kRowsPer];  // cache row of this thread's rows, or -1
      auto locate = [&](int j) {
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int tok = it->r.lo16 + j * kTileN + rbase + kRowStep * i;
          at[i] = -1;
          if (tok < len) {
            const int pg = p.page_shift >= 0 ? tok >> p.page_shift
                                             : (int)fastdiv((uint32_t)tok, p.by_page);
            int64_t page = table[pg];
            if (page < 0 || page >= p.pages) {
              page = 0;
              flag(p.status, kDevBadIndex);
            }
            at[i] = (page * p.hk + it->h) * p.P + (tok - pg * p.P);
          }
        }
      };
      auto load = [&](const uint8_t* codes, const uint8_t* scales, uint4 (&c)[kRowsPer],
                      uint32_t (&b)[kRowsPer]) {
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          c[i] = make_uint4(0, 0, 0, 0);
          b[i] = 0;  // keys past the request: zeros, whatever the cache holds there
          if (at[i] >= 0) {
            c[i] = *reinterpret_cast<const uint4*>(codes + at[i] * (D / 2) + chunk * 16);
            b[i] = *reinterpret_cast<const uint16_t*>(scales + at[i] * (D / 16) + chunk * 2);
          }
        }
      };
      auto store = [&](uint8_t* dst, const uint4 (&c)[kRowsPer], const uint32_t (&b)[kRowsPer]) {
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int row = rbase + kRowStep * i;
          const uint32_t sc = scales2(b[i]);
          const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t fs = __byte_perm(sc, 0, k < 2 ? 0x1010 : 0x3232);
            uint32_t h[4];
            codes8(words[k], h);
            const int c16 = chunk * 4 + k;
            *reinterpret_cast<uint4*>(dst + (c16 >> 3) * (128 * 128) + row * 128 +
                                      (((c16 & 7) ^ (row & 7)) << 4)) =
                make_uint4(h2mul(h[0], fs), h2mul(h[1], fs), h2mul(h[2], fs), h2mul(h[3], fs));
          }
        }
      };
      locate(it->t0);
      load(p.kc, p.ks, ck, bk);
      load(p.vc, p.vs, cv, bv);
      for (int j = it->t0; j < it->t1; ++j, ++n) {
        const int st = n & 1;
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        if (j + 1 < it->t1) locate(j + 1);
        if (!(ok = wait_warp(&bar.k_free[st], par))) break;
        store(sk + st * kTile, ck, bk);
        fence_smem_async();
        mbar_arrive(&bar.k_full[st]);
        if (j + 1 < it->t1) load(p.kc, p.ks, ck, bk);
        if (!(ok = wait_warp(&bar.v_free[st], par))) break;
        store(sv + st * kTile, cv, bv);
        fence_smem_async();
        mbar_arrive(&bar.v_full[st]);
        if (j + 1 < it->t1) load(p.vc, p.vs, cv, bv);
      }
    }
  } else {
    // ==== MMAs: one thread =======================================================
    fewer_registers<kRegsMma>();
    if (warp == 12) {
      constexpr uint32_t kQK = mma_desc(128, false), kPV = mma_desc(D, true);
      const uint32_t dq = smem_addr(sq) >> 4, dk = smem_addr(sk) >> 4, dv = smem_addr(sv) >> 4;
      auto qk = [&](int tile, int st) {
        uint32_t a = dq + (kTile >> 4) * tile, b = dk + (kTile >> 4) * st;
        asm volatile("" : "+r"(a), "+r"(b));  // the steps' addresses are added here, not kept
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // 16 values = 32 bytes along a row; 64 values per panel
          const uint32_t o = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
          mma_ss(t_s(tile), smem_desc(a + o, 0), smem_desc(b + o, 0), kQK, k > 0);
        }
        mma_commit(&bar.s_full[tile]);
      };
      auto pv = [&](int tile, int st, bool add) {
        uint32_t b = dv + (kTile >> 4) * st, a = t_s(tile);
        asm volatile("" : "+r"(a), "+r"(b));
#pragma unroll
        for (int k = 0; k < kTileN / 16; ++k)  // 16 keys = two atoms of 8 rows
          mma_ts(t_o(tile), a + 8 * k, smem_desc(b + (2048 >> 4) * k, 128 * 128), kPV,
                 add || k > 0);
      };
      uint32_t n = 0;  // tiles done
      uint32_t qphase = 0, q1phase = 0, pphase = 0, p1phase = 0;
      bool ok = true;
      while (ok && next(it)) {
        const int tiles = it->t1 - it->t0;
        const bool two = it->rows > kRowsTile;
        if (lane == 0) ok = [&]() -> bool {
          if (!wait(&bar.q_full[0], qphase)) return false;
          if (two && !wait(&bar.q_full[1], q1phase)) return false;
          if (!wait(&bar.k_full[n & 1], (n >> 1) & 1)) return false;
          fence_after();
          qk(0, n & 1);
          if (two) qk(1, n & 1);
          mma_commit(&bar.k_free[n & 1]);
          for (int j = 0; j < tiles; ++j) {
            const uint32_t nj = n + j;
            const int st = nj & 1, sn = st ^ 1;
            const bool more = j + 1 < tiles;
            if (!wait(&bar.v_full[st], (nj >> 1) & 1)) return false;
            if (!wait(&bar.p_full[0], (pphase + j) & 1)) return false;
            fence_after();
            pv(0, st, j > 0);
            if (more) {
              if (!wait(&bar.k_full[sn], ((nj + 1) >> 1) & 1)) return false;
              fence_after();
              qk(0, sn);
            } else {
              mma_commit(&bar.o_done[0]);
            }
            if (two) {
              if (!wait(&bar.p_full[1], (p1phase + j) & 1)) return false;
              fence_after();
              pv(1, st, j > 0);
              if (!more) mma_commit(&bar.o_done[1]);
            }
            mma_commit(&bar.v_free[st]);
            if (more) {
              if (two) qk(1, sn);
              mma_commit(&bar.k_free[sn]);
            }
          }
          return true;
        }();
        ok = __shfl_sync(kAll, ok, 0);
        n += tiles;
        qphase ^= 1;
        pphase += tiles;
        if (two) {
          q1phase ^= 1;
          p1phase += tiles;
        }
      }
      // nothing of this CTA's is in flight when its tensor memory is freed
      if (lane == 0) {
        mma_commit(&bar.end);
        const long long t0 = clock64();
        while (!mbar_try(&bar.end, 0) && clock64() - t0 < kWaitCycles) {
        }
      }
      __syncwarp();
    } else if (warp == 13) {
      if (lane == 0) {
        Walk walk;
        walk.start(p, first, last, s_b0, s_off);
        bool more = true;
        for (uint32_t i = 0; more; ++i) {
          if (!wait(&bar.item_free[i % kItems], ((i / kItems) & 1) ^ 1)) break;
          Item x;
          more = walk.next(p, x);
          if (!more) x.t1 = 0;
          s_item[i % kItems] = x;
          mbar_arrive(&bar.item_full[i % kItems]);
        }
      }
      __syncwarp();
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 12) tmem_free(tmem, 512);
}

template <int D>
cudaError_t launch_t(const KvAttnParams& p, cudaStream_t st) {
  constexpr size_t smem = Smem<D>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(
      kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(sm_count(), kPrefillMaxCtas);
  return launch_pdl_smem(kv_prefill_kernel<D>, dim3(ctas), dim3(kThreads), smem, st, p, ctas);
}

}  // namespace

cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, cudaStream_t st) {
  return D == 128 ? launch_t<128>(p, st) : launch_t<64>(p, st);
}

}  // namespace nvfp4
