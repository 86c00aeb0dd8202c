// kv_prefill.cu -- attention over a paged KV cache held in NVFP4, for many
// query rows per KV head (prompts): the two products on the tensor cores.
//
// The formula, the exactness of K and V in f16 and the numerics of the softmax
// are those of kv_attn.cu. Here a CTA takes 256 query rows of one KV head as
// two tiles of 128 (M), and walks over the keys 64 at a time:
//   S = Q K^T  (Q, K in shared memory; S fp32 in tensor memory)
//   P = 2^(S f - m + bias), f16, written over S in tensor memory
//   O += P V   (P from tensor memory, V in shared memory; O fp32 in tensor memory)
// Tensor memory: two S of 64 columns per tile, O of D columns per tile: 512
// columns at D = 128. With two S per tile the products of the next 64 keys run
// while the softmax works on these, and the softmax never waits for them.
//
// Warps: 0-3 softmax of tile 0 (thread = row), 4-7 of tile 1, which also load
// the next item's query rows while the last products run; 8-11 dequantise K and V
// into shared memory (128 keys at a time, two buffers each); 12 and 15 issue the
// MMAs of tiles 0 and 1; 13 hands out the items; 14 finds the cache rows of the
// keys (block table). All hand-overs are mbarriers.
//
// K and V are dequantised once per 256 query rows: 128 threads turn 16 bytes of
// codes into 32 f16 values each, in the 128-byte-swizzled layout the tensor
// cores read (K rows along k, V rows along n).
//
// Work split: as in kv_attn.cu, the items' key tiles, and what an item costs beside
// them, are cut into equal runs, one per CTA; an item cut between CTAs is joined by the CTA that takes its last
// ticket, in order.
//
// What bounds it: 4 D flops per query row and key on the tensor cores. 64 keys for
// both tiles take 1600 clocks: 1280 of MMAs (1024 by their flops; with 64 keys per
// product the operands' way out of shared memory sets the rate of Q K^T, 48 clocks
// against 32) and a softmax of 1200 beside them, which wait for one another at times.
// From one item to the next both tiles stand still (queries, first scores, last P V,
// result: about 12000 clocks for an item of 34 key tiles). Prompts of 1500 to 2048
// tokens behind 3000 to 10000 (4 requests, 32 query heads on 8, D = 128; 585 GFLOP): 417
// us, 1.40 PFLOP/s, 73% of the measured cuBLAS rate; one prompt of 8192 tokens: 398 us,
// 1.38 PFLOP/s; one of 300: 26 us, all of it latency. Leaving NaN blocks of V out (put_nan)
// costs 5 us of the 417, and 3% where 32 rows wait for the de-quantisation.
//
// Why 64 keys per product and two S per tile: with one S of 128 columns per tile the
// softmax and the MMAs of a tile take turns and it took 545 us where this form then took
// 515. Why one warpgroup that dequantises: two of them (640 threads) leave the softmax
// 152 registers and took 462 us where one took 413. Why K and V are handed over 128 keys
// at a time: 64 at a time (finer barriers, the same buffers) took 517 us where this took
// 413. Why short loops outside the step: the kernel has to stay in the instruction cache;
// with everything unrolled (195 KB of code, then 87, now 95) it took 497 us where it then
// took 445.
//
// Every wait has a limit: when it runs out the CTA sets NVFP4_DEV_TIMEOUT, its
// other waits return at once, and it frees its tensor memory and ends.
#include "kv_attn.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 512;  // 4 warpgroups
// Registers per thread: the softmax keeps a whole row of scores. Two softmax
// warpgroups, one that dequantises, one that issues: 2 x 184 + 88 + 56 = 4 x 128.
constexpr int kRegsSoftmax = 184, kRegsDequant = 88, kRegsMma = 56;
static_assert(2 * kRegsSoftmax + kRegsDequant + kRegsMma <= 4 * 128, "the block's registers");
constexpr int kTileN = 128;    // keys per tile (dequantised together)
constexpr int kStepN = 64;     // keys per product
constexpr int kRowsTile = 128, kRowsItem = 256;
constexpr int kItems = 4;      // items handed out ahead
// What an item costs beside its tiles (queries, first scores, result), in tiles: without
// it the CTA whose run holds the most short items ends last (one prompt of 8192 tokens:
// 510 us with 0, 441 with 2, 405 with 4, 413 with 6; 16 prompts of 512: 102, 101, 92, 98).
constexpr int kItemCost = 4;
constexpr long long kWaitCycles = 2000000000;  // about a second
constexpr uint32_t kNegInf = 0xFF800000u;

__device__ __forceinline__ bool wait_long(uint64_t* b, uint32_t parity, volatile int* dead,
                                          int32_t* status) {
  const long long t0 = clock64();
  while (!mbar_try(b, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > kWaitCycles) {
      *dead = 1;
      flag(status, kDevTimeout);
      return false;
    }
  }
  return true;
}

// 0xFFFF in every half of an f16x2 that is a number.
__device__ __forceinline__ uint32_t numbers2(uint32_t a) {
  uint32_t r;
  asm("set.eq.u32.f16x2 %0, %1, %1;" : "=r"(r) : "r"(a));
  return r;
}

struct Bars {
  uint64_t q_full[2];
  uint64_t s_full[2][2], p_full[2][2];  // [tile][S buffer]
  uint64_t o_done[2];                   // one phase per P V
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t item_full[kItems], item_free[kItems];
  uint64_t rows_full[kItems], rows_free[kItems];  // cache rows of a tile's keys
  uint64_t end;
};

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;  // bytes of a 128 x D f16 tile
  static constexpr int kOut = 8 * 32 * 64;       // 32 rows x 32 bf16 per softmax warp
  static constexpr size_t kBytes = 2 * kTile + 4 * (size_t)kTile + kOut + 1024;  // + alignment
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
  const int hi = r.len - r.n + (int)fastdiv((uint32_t)last, p.by_group) + 1;
  int begin = 0;
  if (p.window > 0) {
    const int low = r.len - r.n + (int)fastdiv((uint32_t)(pt * kRowsItem), p.by_group) + 1 -
                    min(p.window, r.len);
    begin = max(0, low - r.lo16) / kTileN;
  }
  return {begin, max(1, (hi - r.lo16 + kTileN - 1) / kTileN - begin)};
}
// A run is counted in units: kItemCost for the item (nothing runs in them), then one
// per tile. Those of the request's row blocks first, first + step, ..., all heads:
__device__ __forceinline__ int64_t request_units(const KvAttnParams& p, const Request& r,
                                                 int first, int step) {
  int64_t c = 0;
  const int n = row_blocks(p, r);
#pragma unroll 1
  for (int pt = first; pt < n; pt += step) c += block_tiles(p, r, pt).count + kItemCost;
  return c * p.hk;
}

// Inclusive sum over the lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

struct Item {
  Request r;
  int b, h, row0, rows;
  float kg, vg;   // outer scales of K and V
  int t0, t1;     // this CTA's tiles, counted from key lo16
  int c0, c1;     // the CTAs that share it
  int nan_lo, nan_hi;  // keys of those tiles where V has a NaN scale lie in [nan_lo, nan_hi]
};

// The items of this CTA's run [pos, last) of units, in the same order in every
// warp: row blocks inside heads inside requests.
struct Walk {
  int64_t pos, last, run;
  int64_t skip;  // units before pos, counted from (b, h, pt)
  int b, h, pt, blocks;
  Request r;
  __device__ __forceinline__ void start(const KvAttnParams& p, int64_t first, int64_t end,
                                        int64_t per_cta, int b0, int64_t off, int64_t per_head) {
    pos = first;
    run = per_cta;
    last = end;
    b = b0;
    bool bad;
    r = many_rows(p, b, bad);
    blocks = row_blocks(p, r);
    h = (int)(off / per_head);
    skip = off - h * per_head;
    pt = 0;
  }
  __device__ __forceinline__ bool next(const KvAttnParams& p, Item& it) {
#pragma unroll 1
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
      const int units = t.count + kItemCost;
      if (skip >= units) {
        skip -= units;
        ++pt;
        continue;
      }
      const int64_t item = pos - skip;
      const int from = (int)skip, count = (int)min((int64_t)units - skip, last - pos);
      pos += count;
      skip += count;
      if (from + count <= kItemCost) continue;  // none of its tiles
      it.r = r;
      it.b = b;
      it.h = h;
      it.row0 = pt * kRowsItem;
      it.rows = min(kRowsItem, r.n * p.G - it.row0);
      it.t0 = t.begin + max(from - kItemCost, 0);
      it.t1 = t.begin + from + count - kItemCost;
      it.c0 = (int)((item + kItemCost) / run);
      it.c1 = (int)((item + units - 1) / run);
      it.nan_lo = INT32_MAX;
      it.nan_hi = -1;
      const SliceScale ks = slice_scale(p.k_amax[h], p.M), vs = slice_scale(p.v_amax[h], p.M);
      if (ks.bad || vs.bad) flag(p.status, NVFP4_DEV_BAD_AMAX_BIT);
      it.kg = ks.g;
      it.vg = vs.g;
      return true;
    }
    return false;
  }
};

// Loads the item's query rows of one warp (rows 32 w .. + 31 of tile `tile`) into the
// tile's shared memory, LPR lanes to a row, and scales them to f16 in place, a lane to a
// row; returns the score factor of this lane's row. Short loops: code that runs once per
// item comes from far away (unrolled, with the rows in registers and their maxima by way
// of shuffles, it took 9700 clocks an item).
template <int D>
__device__ __forceinline__ float load_queries(const KvAttnParams& p, const Item& x, uint8_t* dst,
                                              int tile, int w, int lane) {
  constexpr int LPR = D / 8, kPer = 32 / LPR;
  const int rows = x.r.n * p.G, first_row = x.row0 + tile * kRowsTile + w * 32;
  dst += w * 32 * 128;
  // chunk c of row i
  auto at = [&](int i, int c) {
    return dst + (c >> 3) * (128 * 128) + i * 128 + (((c & 7) ^ (i & 7)) << 4);
  };
  {
    const int c = lane % LPR;
    const uint16_t* from = p.q + (int64_t)x.r.q0 * p.q_st + (int64_t)(x.h * p.G) * D + c * 8;
#pragma unroll 4
    for (int j = 0; j < 32; j += kPer) {
      const int i = j + lane / LPR, rr = first_row + i;
      const int tk = (int)fastdiv((uint32_t)rr, p.by_group), hh = rr - tk * p.G;
      const bool in = rr < rows;  // the others become zeros
      cp_async16_zfill(at(i, c), in ? from + (int64_t)tk * p.q_st + hh * D : from, in ? 16 : 0);
    }
  }
  cp_async_commit();
  cp_async_wait<0>();
  __syncwarp();
  uint32_t m = 0;
#pragma unroll 4
  for (int c = 0; c < LPR; ++c)
    m = max(m, absmax_bits4(*reinterpret_cast<const uint4*>(at(lane, c))));
  if (m >= 0x7F80u) flag(p.status, NVFP4_DEV_NONFINITE_INPUT_BIT);
  // 2^e brings the row's largest element to [2^13, 2^14)
  const int e = min(max(13 - ((int)(m >> 7) - 127), -126), 126);
  float up = __uint_as_float((uint32_t)(127 + e) << 23);
  float f = p.scale * kLog2e * x.kg * __uint_as_float((uint32_t)(127 - e) << 23);
  if (f < 0.0f) f = -f, up = -up;   // the running maximum needs f > 0, and a masked
  f = fmaxf(f, 1.17549435e-38f);    // score (-inf) must stay -inf times f
#pragma unroll 4
  for (int c = 0; c < LPR; ++c) {
    uint4* q = reinterpret_cast<uint4*>(at(lane, c));
    const uint4 v = *q;
    *q = make_uint4(pack_f16x2(bf16_lo(v.x) * up, bf16_hi(v.x) * up),
                    pack_f16x2(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                    pack_f16x2(bf16_lo(v.z) * up, bf16_hi(v.z) * up),
                    pack_f16x2(bf16_lo(v.w) * up, bf16_hi(v.w) * up));
  }
  fence_smem_async();
  __syncwarp();
  return f;
}

// Record of CTA c's part of an item that begins in CTA c0.
__device__ __forceinline__ float* prefill_record(const KvAttnParams& p, int c, int c0) {
  return p.part + (int64_t)(c * 2 + (c == c0 ? 1 : 0)) * kPrefillRecord;
}
// Weight of CTA c's part in row ri of the whole, whose maximum is m.
__device__ __forceinline__ float part_weight(const KvAttnParams& p, int c, int c0, int ri,
                                             float m) {
  const float mc = __ldcg(prefill_record(p, c, c0) + kRowsItem * 128 + ri);
  return mc == __uint_as_float(kNegInf) ? 0.0f : ex2(mc - m);
}

// The cache row of a request's key.
__device__ __forceinline__ uint32_t cache_row(const KvAttnParams& p, const int32_t* table, int h,
                                              int key) {
  const int pg = p.page_shift >= 0 ? key >> p.page_shift : (int)fastdiv((uint32_t)key, p.by_page);
  int64_t page = table[pg];
  if (page < 0 || page >= p.pages) {
    page = 0;
    flag(p.status, kDevBadIndex);
  }
  return (uint32_t)((page * p.hk + h) * p.P + (key - pg * p.P));
}

// NaN into the output columns (tensor memory, at `to`) of the 16-value blocks of V whose
// scale is NaN in a key that this lane's row sees: keys [low, low + span) among the item's
// nan_lo .. nan_hi. Such blocks are left out of the product, where they would reach every
// row as 0 x NaN. For whole warps; `done` is the barrier of the item's last product.
template <int D>
__device__ __noinline__ bool put_nan(const KvAttnParams& p, const Item& x, int low, uint32_t span,
                                     uint32_t to, uint64_t* done, uint32_t parity,
                                     volatile int* dead) {
  const int lane = threadIdx.x & 31;
  const int32_t* table = p.table + (int64_t)x.b * p.cols;
  uint32_t seen = 0;  // a bit per block
#pragma unroll 1
  for (int first = x.nan_lo; first <= x.nan_hi; first += 32) {
    uint32_t bits = 0;
    if (first + lane <= x.nan_hi) {
      const uint8_t* at = p.vs + (uint64_t)cache_row(p, table, x.h, first + lane) * (D / 16);
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) bits |= (uint32_t)((at[i] & 0x7F) == 0x7F) << i;
    }
    uint32_t some = __ballot_sync(kAll, bits != 0);
    while (some) {
      const int src = __ffs(some) - 1;
      const uint32_t b = __shfl_sync(kAll, bits, src);
      if ((uint32_t)(first + src - low) < span) seen |= b;
      some &= some - 1;
    }
  }
  if (!__all_sync(kAll, wait_long(done, parity, dead, p.status))) return false;
  fence_after();
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t o[16];
    tmem_ld16(to + 16 * c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = seen >> c & 1 ? 0x7FFFFFFFu : o[i];
    tmem_st16(to + 16 * c, o);
  }
  tmem_wait_st();
  return true;
}

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
  __shared__ int64_t s_off, s_per_head;
  __shared__ Walk s_walk;
  __shared__ Item s_item[kItems];
  // first cache row of every 16 keys of a tile: 16 neighbours never leave a page
  __shared__ uint32_t s_rows[kItems][kTileN / 16];
  constexpr int kTile = Smem<D>::kTile;
  uint8_t* base = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint8_t* sq = base;               // [2] Q tiles
  uint8_t* sk = base + 2 * kTile;   // [2] K tiles
  uint8_t* sv = base + 4 * kTile;   // [2] V tiles
  uint8_t* so = base + 6 * kTile;   // results on their way out

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);

  // ---- this CTA's run -------------------------------------------------------
  // `per` threads to a request (one to several requests where there are many)
  int per = 32;
  while (per > 1 && (int64_t)p.B * per > kThreads) per >>= 1;
  const int share = (p.B - 1) / (kThreads / per) + 1;
  const int rb0 = min(tid / per * share, p.B), rb1 = min(rb0 + share, p.B);
  int64_t mine = 0;
#pragma unroll 1
  for (int b = rb0; b < rb1; ++b) {
    bool bad;
    const Request r = many_rows(p, b, bad);
    if (bad && blockIdx.x == 0) flag(p.status, kDevBadIndex);
    mine += request_units(p, r, tid % per, per);
  }
  for (int d = per >> 1; d > 0; d >>= 1) mine += __shfl_xor_sync(kAll, mine, d);
  if (tid % per != 0) mine = 0;  // the group's first thread has the sum
  int64_t incl = warp_scan(mine);
  if (lane == 31) s_scan[warp] = incl;
  if (tid == 0) {
    s_dead = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 4);
      mbar_init(&bar.o_done[i], 1);
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.k_free[i], 2);  // both issuing warps
      mbar_init(&bar.v_free[i], 2);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&bar.s_full[i][j], 1);
        mbar_init(&bar.p_full[i][j], 4);
      }
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_free[i], 15);  // softmax, dequantising, issuing, row-finding warps
      mbar_init(&bar.rows_full[i], 1);
      mbar_init(&bar.rows_free[i], 4);
    }
    mbar_init(&bar.end, 2);
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
#pragma unroll 1
    for (int b = rb0; b < rb1; ++b) {
      bool bad;
      const int64_t c = share == 1 ? mine : request_units(p, many_rows(p, b, bad), 0, 1);
      if (first < at + c) {
        s_b0 = b;
        s_off = first - at;
        s_per_head = c / p.hk;
        break;
      }
      at += c;
    }
  }

  // ---- requests without keys -------------------------------------------------
#pragma unroll 1
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    bool bad;
    const Request r = many_rows(p, b, bad);
    if (r.n == 0 || r.len > 0) continue;
    const int64_t rows = (int64_t)r.n * p.hq;
#pragma unroll 1
    for (int64_t i = tid; i < rows * (D / 8); i += kThreads)
      reinterpret_cast<uint4*>(p.out)[(int64_t)r.q0 * p.hq * (D / 8) + i] = make_uint4(0, 0, 0, 0);
    if (p.lse)
#pragma unroll 1
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
    return mbar_try(b, parity) || wait_long(b, parity, &s_dead, p.status);
  };
  // the same for a whole warp, whose lanes go on together
  auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(kAll, wait(b, parity));
  };

  // The item a warp is at: handed out by warp 13, one after the other, by way of
  // a ring; t1 = 0 ends the run. Asking for the next one gives the last one back.
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
    uint32_t n = 0;  // steps of 64 keys done by this tile
    // The item being worked on: what its result needs, too, which is written when the
    // next item's query rows have been loaded (while the last P V runs).
    float m = 0.0f, l = 0.0f, f = 0.0f, vg = 0.0f;
    int row0 = 0, rows = 0, tk = 0, q0 = 0, h_now = 0, c0 = 0, c1 = 0;
    bool live = false, open = false, ok = true;
    while (ok) {
      const bool have = next(it), mine_now = have && tile * kRowsTile < it->rows;
      // (the products with the query rows that were there are done: their last scores
      // have been seen)
      if (mine_now) {
        f = load_queries<D>(p, *it, sq + tile * kTile, tile, warp & 3, lane);
        if (lane == 0) mbar_arrive(&bar.q_full[tile]);
      }
      if (open) {
        open = false;
        // -- the last item's result: the whole row, or a record of this CTA's part of it
        if (!(ok = wait_warp(&bar.o_done[tile], (n - 1) & 1))) break;
        fence_after();
        float s[32];
        const int ri = tile * kRowsTile + row;
        bool write = true;
        if (c0 != c1) {
          // [D / 4][256 rows][4], then maxima and sums
          float* rec = prefill_record(p, blockIdx.x, c0);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            tmem_ld32(to + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s));
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              reinterpret_cast<float4*>(rec)[(8 * c + i) * kRowsItem + ri] =
                  make_float4(s[4 * i], s[4 * i + 1], s[4 * i + 2], s[4 * i + 3]);
          }
          rec[kRowsItem * 128 + ri] = m;
          rec[kRowsItem * 129 + ri] = l;
          // a row is written by the same warp of every CTA: a ticket per warp
          __threadfence();
          __syncwarp();
          uint32_t* ticket = p.tickets + kAttnMaxCtas + 8 * c0 + warp;
          uint32_t mine_ticket = 0;
          if (lane == 0) mine_ticket = atomicAdd(ticket, 1u);
          write = __shfl_sync(kAll, mine_ticket, 0) == (uint32_t)(c1 - c0);
          if (write) {  // the last CTA to get here joins the parts, in order
            __threadfence();
            if (lane == 0) *ticket = 0;
            m = __uint_as_float(kNegInf), l = 0.0f;
#pragma unroll 1
            for (int c = c0; c <= c1; ++c)
              m = fmaxf(m, __ldcg(prefill_record(p, c, c0) + kRowsItem * 128 + ri));
#pragma unroll 1
            for (int c = c0; c <= c1; ++c)
              l += part_weight(p, c, c0, ri, m) *
                   __ldcg(prefill_record(p, c, c0) + kRowsItem * 129 + ri);
          }
        }
        if (write) {
          // Rows leave four lanes to a row, 64 bytes at a time, by way of shared memory
          // (a thread's own row would go out in 16-byte pieces, half a sector each).
          const float fo = l == 0.0f ? 0.0f : vg / l;
          uint8_t* mine_so = so + warp * (32 * 64);
          // rows of the output past this request's first, -1 where there is none
          const int to_row = live ? tk * p.hq + h_now * p.G + (row0 + row - tk * p.G) : -1;
          if (live && p.lse)
            p.lse[(int64_t)q0 * p.hq + to_row] =
                l == 0.0f ? __uint_as_float(kNegInf) : (m - kBias + log2f(l)) * kLn2;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            if (c0 == c1) {
              tmem_ld32(to + 32 * c, reinterpret_cast<uint32_t(&)[32]>(s));
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = 0.0f;
#pragma unroll 1
              for (int part = c0; part <= c1; part += 2) {  // two parts' loads in flight
                float4 x[2][8];
                float wt[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int from = min(part + k, c1);
                  const float4* q = reinterpret_cast<const float4*>(prefill_record(p, from, c0)) +
                                    8 * c * kRowsItem + ri;
#pragma unroll
                  for (int i = 0; i < 8; ++i) x[k][i] = __ldcg(q + i * kRowsItem);
                  wt[k] = part + k > c1 ? 0.0f : part_weight(p, from, c0, ri, m);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int i = 0; i < 8; ++i) {  // (a weight of 0 leaves a NaN)
                    s[4 * i] = __fmaf_rn(x[k][i].x, wt[k], s[4 * i]);
                    s[4 * i + 1] = __fmaf_rn(x[k][i].y, wt[k], s[4 * i + 1]);
                    s[4 * i + 2] = __fmaf_rn(x[k][i].z, wt[k], s[4 * i + 2]);
                    s[4 * i + 3] = __fmaf_rn(x[k][i].w, wt[k], s[4 * i + 3]);
                  }
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* x = s + 8 * i;
              *reinterpret_cast<uint4*>(mine_so + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(pack_bf16x2(x[0] * fo, x[1] * fo), pack_bf16x2(x[2] * fo, x[3] * fo),
                             pack_bf16x2(x[4] * fo, x[5] * fo), pack_bf16x2(x[6] * fo, x[7] * fo));
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int row32 = q * 8 + (lane >> 2);
              const int at = __shfl_sync(kAll, to_row, row32);
              const uint4 v = *reinterpret_cast<const uint4*>(
                  mine_so + row32 * 64 + (((lane & 3) ^ ((row32 >> 1) & 3)) << 4));
              if (at >= 0)
                reinterpret_cast<uint4*>(p.out)[((int64_t)q0 * p.hq + at) * (D / 8) + 4 * c +
                                                (lane & 3)] = v;
            }
            __syncwarp();
          }
        }
      }
      if (!have) break;
      if (!mine_now) continue;
      const Request r = it->r;
      row0 = it->row0 + tile * kRowsTile, rows = r.n * p.G;
      tk = (int)fastdiv((uint32_t)(row0 + row), p.by_group);
      live = row0 + row < rows;
      q0 = r.q0, h_now = it->h, vg = it->vg, c0 = it->c0, c1 = it->c1;
      // the row sees keys [low, low + span)
      const int lim = live ? r.len - r.n + tk + 1 : 0;
      const int low = p.window > 0 ? lim - min(p.window, r.len) : 0;
      const uint32_t span = (uint32_t)max(lim - low, 0);
      // keys in [safe_lo, safe_hi) are seen by every live row of the tile
      const int last_row = min(row0 + kRowsTile, rows) - 1;
      const int safe_hi = r.len - r.n + (int)fastdiv((uint32_t)row0, p.by_group) + 1;
      const int safe_lo = p.window > 0 ? r.len - r.n + (int)fastdiv((uint32_t)last_row, p.by_group) +
                                             1 - min(p.window, r.len)
                                       : 0;
      m = __uint_as_float(kNegInf), l = 0.0f;
      const int steps = 2 * (it->t1 - it->t0);
      int key0 = r.lo16 + it->t0 * kTileN;

      for (int j = 0; j < steps; ++j, ++n, key0 += kStepN) {
        const uint32_t sb = n & 1;
        if (!(ok = wait_warp(&bar.s_full[tile][sb], (n >> 1) & 1))) break;
        fence_after();
        uint32_t s[2][32];
        tmem_ld32(ts + kStepN * sb, s[0]);
        tmem_ld32(ts + kStepN * sb + 32, s[1]);
        tmem_wait_ld();
        if (key0 + kStepN > safe_hi || key0 < safe_lo) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((uint32_t)(key0 - low + 32 * c + i) >= span) s[c][i] = kNegInf;
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[0][i]);
#pragma unroll
        for (int i = 4; i < 64; i += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (i + 2 * q + 1 < 64)
              mx[q] = fmax3(mx[q], __uint_as_float(s[(i + 2 * q) >> 5][(i + 2 * q) & 31]),
                            __uint_as_float(s[(i + 2 * q + 1) >> 5][(i + 2 * q + 1) & 31]));
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * f;
        if (__any_sync(kAll, top > m + kSlack)) {
          const float mn = fmaxf(m, top);
          const float a = m == __uint_as_float(kNegInf) ? 0.0f : ex2(m - mn);
          m = mn;
          l *= a;
          if (j > 0) {
            // the previous P V has to be done (the one before it is: the scores here
            // were asked for behind it)
            if (!(ok = wait_warp(&bar.o_done[tile], (n - 1) & 1))) break;
            fence_after();
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
        f2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            f2 x = f2_fma(make_float2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])),
                          ff, cc);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            sum[i & 1] = __fadd2_rn(sum[i & 1], x);
            h[i] = pack_f16x2(x.x, x.y);
          }
          tmem_st16(ts + kStepN * sb + 16 * c, h);
        }
        tmem_wait_st();
        // A phase's parity does not tell it from the one two before. Scores n say
        // that P V n - 2 is done, and P V n cannot start before this arrival: so the
        // last step of an item sees P V n - 1 done here, and n behind the loop.
        if (j == steps - 1 && !(ok = wait_warp(&bar.o_done[tile], (n - 1) & 1))) break;
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[tile][sb]);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      // (a P V of the item's last tile is done: its V was stored and looked at)
      if (ok && it->nan_hi >= 0)
        ok = put_nan<D>(p, *it, low, span, to, &bar.o_done[tile], (n - 1) & 1, &s_dead);
      open = true;
    }
  } else if (warp < 12) {
    // ==== dequantise ============================================================
    fewer_registers<kRegsDequant>();
    // thread: rows 8 w + (lane & 7) + 32 i of a tile, 16-byte chunk lane / 8 of the
    // codes (D = 64: rows 16 w + (lane & 15) + 64 i, chunk lane / 16): a quarter
    // warp's stores hit all banks once
    constexpr int kRowsPer = D == 128 ? 4 : 2, kRowStep = D == 128 ? 32 : 64;
    const int w = warp - 8;
    const int rbase = D == 128 ? w * 8 + (lane & 7) : w * 16 + (lane & 15);
    const int chunk = D == 128 ? lane >> 3 : lane >> 4;
    uint32_t n = 0;  // tiles done
    bool ok = true;
    while (ok && next(it)) {
      const int len = it->r.len, t1 = it->t1;
      int tok = it->r.lo16 + it->t0 * kTileN + rbase;  // this thread's first key of a tile
      uint4 ck[kRowsPer], cv[kRowsPer];
      uint32_t bk[kRowsPer], bv[kRowsPer];
      uint32_t at[kRowsPer];   // cache rows of this thread's keys
      bool in[kRowsPer];       // ... that the request has
      auto locate = [&](uint32_t tile_n, int first) -> bool {
        const uint32_t slot = tile_n % kItems;
        if (!wait_warp(&bar.rows_full[slot], (tile_n / kItems) & 1)) return false;
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int row = rbase + kRowStep * i;
          at[i] = s_rows[slot][row >> 4] + (row & 15);
          in[i] = first + kRowStep * i < len;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.rows_free[slot]);
        return true;
      };
      auto load = [&](const uint8_t* codes, const uint8_t* scales, uint4 (&c)[kRowsPer],
                      uint32_t (&b)[kRowsPer]) {
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          c[i] = make_uint4(0, 0, 0, 0);
          b[i] = 0;  // keys past the request: zeros, whatever the cache holds there
          if (in[i]) {
            c[i] = *reinterpret_cast<const uint4*>(codes + (uint64_t)at[i] * (D / 2) + chunk * 16);
            b[i] = *reinterpret_cast<const uint16_t*>(scales + (uint64_t)at[i] * (D / 16) + chunk * 2);
          }
        }
      };
      auto store = [&](uint8_t* dst, const uint4 (&c)[kRowsPer], const uint32_t (&b)[kRowsPer],
                       bool v) {
        uint32_t nan = 0;
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
          const int row = rbase + kRowStep * i;
          uint32_t sc = scales2(b[i]);
          // In P V a NaN block would reach rows that do not see its key, as 0 x NaN: it is
          // left out, and the rows that see it get the NaN at the item's end.
          if (v) {
            const uint32_t number = numbers2(sc);
            sc &= number;
            nan |= ~number;
          }
          const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t fs = __byte_perm(sc, 0, k < 2 ? 0x1010 : 0x3232);
            uint32_t x[4];
            codes8(words[k], x);
            const int c16 = chunk * 4 + k;
            *reinterpret_cast<uint4*>(dst + (c16 >> 3) * (128 * 128) + row * 128 +
                                      (((c16 & 7) ^ (row & 7)) << 4)) =
                make_uint4(h2mul(x[0], fs), h2mul(x[1], fs), h2mul(x[2], fs), h2mul(x[3], fs));
          }
        }
        if (nan) {
          atomicMin(&s_item[(items - 1) % kItems].nan_lo, tok);
          atomicMax(&s_item[(items - 1) % kItems].nan_hi, min(tok + kRowStep * (kRowsPer - 1), len - 1));
        }
        fence_smem_async();
        __syncwarp();
      };
      if (!(ok = locate(n, tok))) break;
      load(p.kc, p.ks, ck, bk);
      load(p.vc, p.vs, cv, bv);
      for (int j = it->t0; j < t1; ++j, ++n, tok += kTileN) {
        const int st = n & 1;
        const uint32_t par = ((n >> 1) & 1) ^ 1;
        const bool more = j + 1 < t1;
        if (more && !(ok = locate(n + 1, tok + kTileN))) break;
        if (!(ok = wait_warp(&bar.k_free[st], par))) break;
        store(sk + st * kTile, ck, bk, false);
        if (lane == 0) mbar_arrive(&bar.k_full[st]);
        if (more) load(p.kc, p.ks, ck, bk);
        if (!(ok = wait_warp(&bar.v_free[st], par))) break;
        store(sv + st * kTile, cv, bv, true);
        if (lane == 0) mbar_arrive(&bar.v_full[st]);
        if (more) load(p.vc, p.vs, cv, bv);
      }
    }
  } else {
    fewer_registers<kRegsMma>();
    if (warp == 12 || warp == 15) {
      // ==== MMAs: one warp per query tile, one thread of it ========================
      const int tile = warp == 12 ? 0 : 1;
      constexpr uint32_t kQK = mma_desc(kStepN, false), kPV = mma_desc(D, true);
      const uint32_t dq = smem_addr(sq + tile * kTile) >> 4;
      const uint32_t dk = smem_addr(sk) >> 4, dv = smem_addr(sv) >> 4;
      const uint32_t ts = t_s(tile), to = t_o(tile);
      // S for 64 keys: half `half` of the K tile in stage st
      auto qk = [&](int st, int half) {
        uint32_t a = dq, b = dk + (kTile >> 4) * st + (kStepN * 128 >> 4) * half;
        asm volatile("" : "+r"(a), "+r"(b));  // the steps' addresses are added here, not kept
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          // 16 values = 32 bytes along a row; 64 values per panel
          const uint32_t o = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
          mma_ss(ts + kStepN * half, smem_desc(a + o, 0), smem_desc(b + o, 0), kQK, k > 0);
        }
        mma_commit(&bar.s_full[tile][half]);
      };
      auto pv = [&](int st, int half, bool add) {
        uint32_t a = ts + kStepN * half;
        uint32_t b = dv + (kTile >> 4) * st + (kStepN * 128 >> 4) * half;
        asm volatile("" : "+r"(a), "+r"(b));
#pragma unroll
        for (int k = 0; k < kStepN / 16; ++k)  // 16 keys = two atoms of 8 rows
          mma_ts(to, a + 8 * k, smem_desc(b + (2048 >> 4) * k, 128 * 128), kPV, add || k > 0);
        mma_commit(&bar.o_done[tile]);
      };
      uint32_t n = 0, mine_n = 0;  // key tiles done, and those of them with this query tile
      uint32_t qphase = 0;
      bool ok = true;
      while (ok && next(it)) {
        const int tiles = it->t1 - it->t0;
        const bool two = it->rows > kRowsTile;
        if (tile == 1 && !two) {
          // follows tile by tile all the same: a barrier's parity only tells
          // neighbouring phases apart
          if (elect_one()) ok = [&]() -> bool {
            for (uint32_t j = n; j < n + tiles; ++j) {
              if (!wait(&bar.k_full[j & 1], (j >> 1) & 1)) return false;
              mbar_arrive(&bar.k_free[j & 1]);
              if (!wait(&bar.v_full[j & 1], (j >> 1) & 1)) return false;
              mbar_arrive(&bar.v_free[j & 1]);
            }
            return true;
          }();
          ok = __all_sync(kAll, ok);
          n += tiles;
          continue;
        }
        if (elect_one()) ok = [&]() -> bool {
          if (!wait(&bar.k_full[n & 1], (n >> 1) & 1)) return false;
          if (!wait(&bar.q_full[tile], qphase)) return false;
          fence_after();
          qk(n & 1, 0);
          qk(n & 1, 1);
          mma_commit(&bar.k_free[n & 1]);
          for (int j = 0; j < tiles; ++j) {
            const uint32_t nj = n + j;
            const int st = nj & 1, sn = st ^ 1;
            const bool more = j + 1 < tiles;
            if (!wait(&bar.v_full[st], (nj >> 1) & 1)) return false;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!wait(&bar.p_full[tile][half], (mine_n + j) & 1)) return false;
              fence_after();
              pv(st, half, j > 0 || half > 0);
              if (more) {
                if (half == 0 && !wait(&bar.k_full[sn], ((nj + 1) >> 1) & 1)) return false;
                fence_after();
                qk(sn, half);
              }
            }
            mma_commit(&bar.v_free[st]);
            if (more) mma_commit(&bar.k_free[sn]);
          }
          return true;
        }();
        ok = __all_sync(kAll, ok);
        n += tiles;
        mine_n += tiles;
        qphase ^= 1;
      }
      // nothing of this warp's is in flight when the tensor memory is freed
      if (elect_one()) {
        mma_commit(&bar.end);
        const long long t0 = clock64();
        while (!mbar_try(&bar.end, 0) && clock64() - t0 < kWaitCycles) {
        }
      }
      __syncwarp();
    } else if (warp == 13) {
      // ==== items ================================================================
      if (lane == 0) s_walk.start(p, first, last, run, s_b0, s_off, s_per_head);
      bool more = true;
      for (uint32_t i = 0; more; ++i) {
        if (!wait_warp(&bar.item_free[i % kItems], ((i / kItems) & 1) ^ 1)) break;
        Item& x = s_item[i % kItems];
        if (lane == 0) {
          more = s_walk.next(p, x);
          if (!more) x.t1 = 0;
          mbar_arrive(&bar.item_full[i % kItems]);
        }
        more = __shfl_sync(kAll, more, 0);
        __syncwarp();
        if (more) {
          // its query rows on their way to L2: they are loaded between two items, where
          // nothing hides their latency
          constexpr int kLines = D * 2 / 128;
          for (int u = lane; u < x.rows * kLines; u += 32) {
            const int rr = x.row0 + u / kLines;
            const int tk = (int)fastdiv((uint32_t)rr, p.by_group);
            const uint16_t* at = p.q + (int64_t)(x.r.q0 + tk) * p.q_st +
                                 (int64_t)(x.h * p.G + rr - tk * p.G) * D + u % kLines * 64;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
          }
          __syncwarp();
        }
      }
    } else if (warp == 14) {
      // ==== cache rows: lane g looks up keys 16 g .. 16 g + 15 of a tile ==========
      uint32_t n = 0;
      bool ok = true;
      while (ok && next(it)) {
        const int32_t* table = p.table + (int64_t)it->b * p.cols;
        const int len = it->r.len, h = it->h, t1 = it->t1;
        int key = it->r.lo16 + it->t0 * kTileN + 16 * lane;
        for (int j = it->t0; j < t1; ++j, ++n, key += kTileN) {
          uint32_t row = 0;
          if (lane < kTileN / 16 && key < len) {
            row = cache_row(p, table, h, key);
          }
          if (!(ok = wait_warp(&bar.rows_free[n % kItems], ((n / kItems) & 1) ^ 1))) break;
          if (lane < kTileN / 16) s_rows[n % kItems][lane] = row;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.rows_full[n % kItems]);
        }
      }
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
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kv_prefill_kernel<D>, smem, ready);
  if (e != cudaSuccess) return e;
  const int ctas = std::min(sm_count(), kPrefillMaxCtas);
  return launch_pdl_smem(kv_prefill_kernel<D>, dim3(ctas), dim3(kThreads), smem, st, p, ctas);
}

}  // namespace

cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, cudaStream_t st) {
  return D == 128 ? launch_t<128>(p, st) : launch_t<64>(p, st);
}

}  // namespace nvfp4
