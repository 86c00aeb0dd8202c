// matmul.cu -- products of block-scaled matrices on tcgen05, grouped by expert.
//
//   NVFP4, MXFP8:        out[t][n] = sum over k of a[t][k] b[e][n][k], e the group of row t
//   weights' gradient:   out[e][n][k] = sum over the rows t of group e of g[n][t] x[k][t]
//
// both as C = F X^T along the operands' rows: 128 rows of F ("features": the weights, or x)
// are the M of a product, up to 256 rows of X ("columns": tokens, or g) its N, any multiple of
// 16, so that a group's last few rows cost what they are and a call of one row reads the weights
// alone. Codes and scales go to the tensor cores as the encoders wrote them; the products apply
// the block scales, the outer scales are applied to the fp32 sums.
//
// One CTA (or a pair) to an SM, 16 warps with a job each: one copies codes by tensor map (and
// hands out the work), one issues the products, six bring the scales, eight take the results. A
// stage of the ring is 128 bytes of codes of every row (256 NVFP4 or 128 MXFP8 values, one
// swizzle line) with its scales; two accumulators that share 64 columns let a tile's products
// begin while the last one's results leave.
//
// Scales. tcgen05 takes them from tensor memory in a layout of its own (32 lines of four rows
// each) that a copy from shared memory fills 512 bytes at a time; in memory a row's scales follow
// one another. NVFP4: a tensor map copies a stage's 16 bytes of 128 rows in one box, and a warp
// turns them in place (a lane reads 16 bytes of its line's four rows and writes them back,
// transposed word by word). Loads by threads, which were there first, cost more than everything
// else together: every 16 bytes are a line of their own to the load unit (dense 8192^3: 303 us;
// 64 bytes of a row at a time 229; by asynchronous copies 256; by tensor map 199). MXFP8 has a
// quarter of them: a lane loads 16 bytes (four stages) of its line's rows, three loads ahead,
// which costs 2%. Rows of scales that are not whole 16 bytes come in two aligned pieces, cut at
// their use, or, where the sum is long enough, are copied to whole ones first.
//
// What bounds it. A 256 x 256 tile of a pair loads 16 KB of F and 16 KB of X per CTA and stage,
// which its products take 512 clocks for (at 16384 NVFP4 or 8192 MXFP8 operations a clock and SM);
// the way from L2 gives an SM about 50 bytes a clock, 660 clocks, and both share the port of shared
// memory. A single CTA's 128 x 256 tile needs 48 KB a stage (NVFP4 8192^3: 205 us without any
// products, pairs 184). Measured, operations a second in the device's time: dense 8192^3 NVFP4
// 5.9 PFLOP/s (3.1 times the measured cuBLAS bf16 rate), MXFP8 3.6 (1.9 times). Where columns are
// few the weights' bytes bound it: 64 experts of 2048 x 7168, 90 rows, 61 us, 84% of the copy
// rate; 16384 ragged rows 126 us (77% of the copy rate, 3.8 PFLOP/s). Weights' gradients write as
// much as they read and their sums are short: 16 experts of 2048 x 7168, 16384 rows, 188 us (2.6
// PFLOP/s), of which the results' way out is 20 us (the change of accumulators is 700 to 1000
// clocks a tile of 8 stages, but products that do not wait for it gain 3 us). These are times at
// the full clock, 2070 MHz: for seconds on end the power limit holds weights' gradients at 1640
// MHz (213 us) and the ragged NVFP4 rows at 1720 (136). Small calls take 6 to 13 us, most of it
// the way to the first copy (cold code and constants, 2 us), DRAM latency and the results.
//
// Results. A lane holds a feature's. Of a product over tokens the features are neighbours in
// memory: lanes swap halves with a shuffle and store 4 bytes. That is nine instructions for two
// values, which a tile of 8 stages has no time for (5800 of its 6700 clocks). A weights' gradient's
// features may be either operand's rows: g's, so that a lane's results are a row's, which go to
// shared memory 16 bytes at a time and leave by tensor map, for one stage of the ring less (199 us
// to 189; 1000 x 544 8.5 to 7.5; sums of 32 stages 147 to 148). Stored from the lanes they took 213
// us in pieces of 32 bytes and 294 of 16; tokens' results by tensor map gain nothing (126 us, MXFP8
// 173 to 175). fp32 results and rows that are not whole 32 bytes go the other way (16 equal experts
// 235 us in fp32, 174 in bf16).
//
// Tried: results turned in shared memory by stmatrix for 16-byte stores (weights' gradient 218 ->
// 248 us: shared memory has no time to spare); every warp finding its own work (220 -> 202 when
// one does it for all); a cluster-scope release for each arrival at the pair's barriers (a stage
// then took 2000 clocks); bands of 1 to 16 column tiles (within 1%).
//
// Every wait has a limit: when it runs out the CTA sets NVFP4_DEV_TIMEOUT, its other waits return
// at once, and it frees its tensor memory and ends.
#include "matmul.h"
#include "tcgen05.cuh"

#include <type_traits>

namespace nvfp4 {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kEpilogueWarps = 8;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kScaleWarps = 6;
constexpr int kThreads = (kEpilogueWarps + 2 + kScaleWarps) * 32;
constexpr int kTileF = 128, kTileC = 256;
constexpr int kStageRow = 128;                 // code bytes of a row in a stage: one swizzle line
constexpr int kFBytes = kTileF * kStageRow;
constexpr int kBox = 128, kBoxSmall = 32;      // rows of one copy
constexpr int kMaxStages = 12;
constexpr int kSmem = 217 * 1024;              // the ring of stages, 1 KB for its alignment
constexpr int kTurn = 2048;                    // bytes of a warp's results on their way out
// Tensor memory: two accumulators of 256 columns that share 64, then the scales of a stage.
constexpr int kAcc1 = 192, kScales = 448;
constexpr int kBand = 8;                       // column tiles of a band
// Columns of a group from which pairs of CTAs pay: 64 experts of 64 rows 91 us alone and 94 in
// pairs, of 96 rows 93 both, of 256 rows 119 and 111.
constexpr int kPairCols = 96;
// Tiles of a call at most: groups in order have 2^26 (the entry points refuse more), groups out of
// order may share rows, and their sums stay at this number.
constexpr int kMaxTiles = 1 << 27;
constexpr double kPadGain = 0.3;               // see launch_matmul
constexpr long long kWaitCycles = 2000000000;  // about a second

__device__ __forceinline__ bool wait_long(uint64_t* b, uint32_t parity, volatile int* dead,
                                          int32_t* status) {
  const long long t0 = clock64();
  while (!mbar_try(b, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > kWaitCycles) {
      *dead = 1;
      flag(status, NVFP4_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The barrier's phase counts one arrival when this thread's copies so far are done.
__device__ __forceinline__ void copies_arrive(uint64_t* b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(b))
               : "memory");
}

// 16 bytes at q (16-byte aligned); those at `end` and after it are 0 and not read.
__device__ __forceinline__ uint4 bytes16(const uint8_t* q, const uint8_t* end) {
  if (q + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(q));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll 1
    for (int i = 0; i < 4; ++i)
      if (q + 4 * j + i < end) w[j] |= (uint32_t)q[4 * j + i] << (8 * i);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes off .. off + 15 of the 32 in lo and hi (off < 16).
__device__ __forceinline__ uint4 window16(uint4 lo, uint4 hi, uint32_t off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t s = 8 * (off & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s),
                    __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}
// x without the bytes from `n` on.
__device__ __forceinline__ uint4 first_bytes(uint4 x, int n) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int m = n - 4 * j;
    w[j] = m >= 4 ? w[j] : m <= 0 ? 0 : w[j] & ((1u << (8 * m)) - 1);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Copies of n columns: large boxes as far as they fill, then one more or, for up to half
// of it, small ones.
struct Boxes {
  int large, count;
  __host__ __device__ __forceinline__ explicit Boxes(int n) {
    const int rest = n % kBox;
    large = n / kBox + (rest > kBox / 2);
    count = large + (rest > kBox / 2 ? 0 : (rest + kBoxSmall - 1) / kBoxSmall);
  }
  __host__ __device__ __forceinline__ int row(int i) const {  // of box i
    return i < large ? i * kBox : large * kBox + (i - large) * kBoxSmall;
  }
  __host__ __device__ __forceinline__ int rows() const { return row(count); }
};

template <int KIND>
struct Kind {
  static constexpr bool kFp4 = KIND == kMatmulNvfp4;
  static constexpr bool kWgrad = KIND == kMatmulMxWgrad;
  static constexpr int kStageK = kFp4 ? 256 : 128;  // values of a row in a stage
  static constexpr int kStepK = kFp4 ? 64 : 32;     // values of a product
  static constexpr int kStageSf = kFp4 ? 16 : 4;    // scale bytes of a row in a stage
  static constexpr int kSfBlock = 128 * kStageSf;   // scale bytes of 128 rows in a stage
  static constexpr int kFetch = 16 / kStageSf;      // stages whose scales are fetched together
  // bytes of the ring of stages (a weights' gradient's results leave through the rest)
  static constexpr int kRing = kSmem - 1024 - (kWgrad ? kEpilogueWarps * kTurn : 0);
};

// How a call is cut: tiles, parts of a tile's sum (where there are more CTAs than tiles), and
// a stage of the ring: features' codes, columns' codes, features' scales, columns' scales (a
// pair's CTA holds half of the columns' codes and all of their scales).
struct Geometry {
  int split, items;
  int c_blocks, sf_at, stage_bytes, stages;
};
// total tiles of at most `most` columns and `stages` stages, for so many CTAs or pairs of CTAs.
// A sum is cut where that saves more than joining its parts costs: a stage takes a CTA about
// 250 ns and 1 ns a column (loads and products of its own tile), the join 4.5 us and 50 ns a
// column (8 rows, 2432 x 16384: 12.5 us cut in 8, 19 whole; 512 rows, 2048 x 7168: 22 us
// cut in 4, 17 whole).
template <int KIND, int CG>
__host__ __device__ __forceinline__ Geometry geometry(int total, int most, int stages, int pairs,
                                                      bool aligned) {
  Geometry g;
  g.split = 1;
  if (total > 0 && 2 * total <= pairs) {
    int split = (int)((uint32_t)pairs / (uint32_t)total);
    if (split > 16) split = 16;
    const int saved = (int)((uint32_t)(stages * (split - 1)) / (uint32_t)split);
    if ((int64_t)saved * (250 + most) > 4500 + 50 * (int64_t)most) g.split = split;
  }
  g.items = total * g.split;
  g.c_blocks = (most + 127) / 128;
  g.sf_at = kFBytes + Boxes(((most + 15) & ~15) / CG).rows() * kStageRow;
  // (NVFP4 scales that are not aligned come as two aligned pieces)
  const int sf = (1 + g.c_blocks) * Kind<KIND>::kSfBlock * (Kind<KIND>::kFp4 && !aligned ? 2 : 1);
  g.stage_bytes = (g.sf_at + sf + 1023) & ~1023;
  g.stages = (int)((uint32_t)Kind<KIND>::kRing / (uint32_t)g.stage_bytes);
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  return g;
}

// What one CTA does at a time: features f0 .. of a group times some of its
// columns, over stages k0 .. k1 - 1 of the sum.
struct Work {
  int g, f0, c0, cols;      // group, first feature, first column, columns
  int f_row, c_row;         // rows of the two matrices
  int k_at;                 // first value of the sum
  int first, steps;         // the sum's first product and the end of its products
  int k0, k1;
  int item, tile, part, parts;  // part -1: no more work
};
constexpr int kWorks = 8;       // pieces of work handed out ahead
constexpr int kTakers = kEpilogueWarps + 1 + kScaleWarps;

// Fills N slots, then empties and refills them in turn until emptying one fails.
template <int N, int I = 0, class Fetch>
__device__ __forceinline__ void fill_ring(Fetch& fetch) {
  if constexpr (I < N) {
    fetch(std::integral_constant<int, I>{});
    fill_ring<N, I + 1>(fetch);
  }
}
template <int N, int I = 0, class Fetch, class Store>
__device__ __forceinline__ bool turn_ring(Fetch& fetch, Store& store) {
  if constexpr (I < N) {
    if (!store(std::integral_constant<int, I>{})) return false;
    fetch(std::integral_constant<int, I>{});
    return turn_ring<N, I + 1>(fetch, store);
  }
  return true;
}
template <int N, class Fetch, class Store>
__device__ __forceinline__ void ring_of(Fetch& fetch, Store& store) {
  fill_ring<N>(fetch);
  while (turn_ring<N>(fetch, store)) {
  }
}

// A place in the ring of stages and the parity of its present turn.
struct Place {
  int st = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) st = 0, turn ^= 1;
  }
};

struct Maps {
  CUtensorMap f, c, c_small;     // codes of the features' and the columns' rows
  CUtensorMap fs, cs, cs_small;  // their scales
  CUtensorMap out;               // a weights' gradient's results
};

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t raw[3][kMaxStages];     // scales of 128 rows as they lie in memory
  uint64_t acc_full, acc_free, end;
  uint64_t work_full[kWorks], work_free[kWorks];
  uint32_t tmem;
  volatile int dead;
  int last;
  int scan[kThreads / 32], most[kThreads / 32];
  Geometry geo;
  Work work[kWorks];
  int tile[kMatmulMaxGroups + 1];  // a group's first tile
  alignas(16) float scale[2][kTileC];  // outer scales of a tile's columns
};

// The epilogue warps' barrier; whether all of them said yes.
__device__ __forceinline__ bool all_of(bool yes) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
               "barrier.cta.red.and.pred.aligned q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((uint32_t)yes), "n"(kEpilogueWarps * 32) : "memory");
  return r != 0;
}

template <int KIND, int CG>
__global__ void __launch_bounds__(kThreads, 1)
matmul_kernel(const __grid_constant__ Maps maps, const MatmulParams p, const Geometry geo_known) {
  using T = Kind<KIND>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared s;
  uint8_t* ring = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  // this CTA of the pair, and the pair (CG = 1: a CTA by itself)
  const int rank = CG == 2 ? (int)cluster_rank() : 0;
  const int pair = (int)blockIdx.x / CG, pairs = (int)gridDim.x / CG;
  const int f_tiles = (p.N + kTileF * CG - 1) / (kTileF * CG);
  const int64_t rows_all = T::kWgrad ? p.K : p.c_rows;
  const bool scan = !T::kWgrad && p.start;  // the tiles are known on the device only

  // Whether 16 scale bytes of a row are aligned in memory.
  const bool sf_aligned = p.sf_stride % 16 == 0;
  // What does not depend on earlier kernels, while they end.
  if (warp == 0) {
    if (lane < kMaxStages) {
      mbar_init(&s.full[lane], 1 + CG * (T::kFp4 ? kScaleWarps / 2 : kScaleWarps));
      mbar_init(&s.empty[lane], 1);
      for (int b = 0; b < 3; ++b) mbar_init(&s.raw[b][lane], sf_aligned ? 1 : 32);
    } else if (lane == kMaxStages) {
      s.dead = 0;
      mbar_init(&s.acc_full, 1);
      mbar_init(&s.acc_free, CG * kEpilogueWarps);
      mbar_init(&s.end, 1);
    } else if (lane - kMaxStages <= kWorks) {
      mbar_init(&s.work_full[lane - kMaxStages - 1], 1);
      mbar_init(&s.work_free[lane - kMaxStages - 1], kTakers);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == kCopyWarp && p.sf_stride > 0 && lane < (T::kFp4 && sf_aligned ? 4 : 2)) {
    // (the large boxes' maps need not be there)
    const CUtensorMap* map =
        lane == 0 ? &maps.f : lane == 1 ? &maps.c_small : lane == 2 ? &maps.fs : &maps.cs_small;
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
  } else if (warp == kMmaWarp) {
    if constexpr (CG == 2) tmem_alloc_pair(&s.tmem, 512);
    else tmem_alloc(&s.tmem, 512);
  }
  __syncwarp();
  if constexpr (CG == 2) cluster_arrive();
  pdl_begin();

  // ---- the groups' tiles -----------------------------------------------------
  // Ragged rows: a thread to `share` groups, then a scan over the threads. Otherwise the
  // host knows the tiles.
  int before = 0, mine = 0;
  const int share = (p.E + kThreads - 1) / kThreads;
  const int e0 = min(tid * share, p.E), e1 = min(e0 + share, p.E);
  if (scan) {
    int most = 0;
    for (int e = e0; e < e1; ++e) {
      int64_t a = p.start[e], b = p.start[e + 1];
      if (a < 0 || b < a || b > rows_all) {
        if (blockIdx.x == 0) flag(p.status, NVFP4_DEV_BAD_INDEX);
        a = b = 0;
      }
      const int cols = (int)(b - a), c_tiles = (cols + p.c_tile - 1) >> p.c_shift;
      if (c_tiles > 0)
        most = max(most, c_tiles == 1 ? cols
                                      : (int)((uint32_t)(cols + c_tiles - 1) / (uint32_t)c_tiles));
      s.tile[e] = mine;
      mine = min(mine + c_tiles * f_tiles, kMaxTiles);
    }
    int incl = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl = min(incl + o, kMaxTiles);
    }
    before = __shfl_up_sync(kAll, incl, 1);
    if (lane == 0) before = 0;
    most = __reduce_max_sync(kAll, most);
    if (lane == 31) s.scan[warp] = incl;
    if (lane == 0) s.most[warp] = most;
  }
  fence_before();
  __syncthreads();
  fence_after();
  if constexpr (CG == 2) cluster_wait();  // the other CTA's barriers are there
  if (scan) {
    int total = 0, most = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before = min(before + s.scan[w], kMaxTiles);
      total = min(total + s.scan[w], kMaxTiles);
      most = max(most, s.most[w]);
    }
    for (int e = e0; e < e1; ++e) s.tile[e] = min(s.tile[e] + before, kMaxTiles);
    if (tid == 0) {
      s.tile[p.E] = total;
      s.geo = geometry<KIND, CG>(total, most, (int)((p.K + T::kStageK - 1) / T::kStageK), pairs,
                                 sf_aligned);
    }
    __syncthreads();
  }
  const Geometry geo = scan ? s.geo : geo_known;
  const int split = geo.split, items = geo.items, c_blocks = geo.c_blocks, sf_at = geo.sf_at;
  const int stage_bytes = geo.stage_bytes, stages = geo.stages;
  const uint32_t tmem = s.tmem;

  // 32-bit unsigned divisions only, and none where there is one of a kind: what a call
  // that fits the SMs once pays before its first copy.
  auto work_of = [&](int item, Work& w) -> bool {
    w.item = w.tile = item;
    w.part = 0;
    if (split > 1) {
      w.tile = (int)((uint32_t)item / (uint32_t)split);
      w.part = item - w.tile * split;
    }
    int lo = 0, ft = w.tile;
    if (scan) {
      int hi = p.E;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.tile[mid] <= w.tile) lo = mid;
        else hi = mid;
      }
      ft -= s.tile[lo];
    } else if (T::kWgrad) {
      lo = (int)fastdiv((uint32_t)w.tile, p.by_tiles);
      ft -= lo * p.tiles;
    }
    w.g = lo;
    int row = 0, rows = (int)rows_all;
    if (p.start) {
      row = __ldg(p.start + lo);
      rows = __ldg(p.start + lo + 1) - row;
    }
    if (T::kWgrad && (row < 0 || rows < 0 || rows > rows_all - row || (row | rows) % 32 != 0)) {
      flag(p.status, NVFP4_DEV_BAD_INDEX);
      return false;
    }
    const int cols = T::kWgrad ? p.C : rows;
    w.c0 = 0;
    w.cols = cols;
    if (cols > p.c_tile) {
      const uint32_t c_tiles = (uint32_t)(cols + p.c_tile - 1) >> p.c_shift;
      uint32_t size = ((uint32_t)cols + c_tiles - 1) / c_tiles;
      if (T::kWgrad) size = (size + 31) & ~31u;  // (a box of results is of one tile)
      // bands of column tiles, a band's columns first
      uint32_t band = 0, in = (uint32_t)ft, wide = c_tiles;
      if (c_tiles > kBand) {
        band = in / (uint32_t)(kBand * f_tiles);
        in -= band * (uint32_t)(kBand * f_tiles);
        wide = min((uint32_t)kBand, c_tiles - band * kBand);
      }
      ft = (int)(in / wide);
      w.c0 = (int)((band * kBand + in - (uint32_t)ft * wide) * size);
      w.cols = min((int)size, cols - w.c0);
    }
    w.f0 = (ft * CG + rank) * kTileF;
    // A weights' gradient sums over values `row` on, in stages that begin at multiples of 128
    // (whole words of scales): the first stage's products in front of it are left out.
    const int skip = T::kWgrad ? row & (T::kStageK - 1) : 0;
    const int sum = T::kWgrad ? (rows > 0 ? rows + skip : 0) : (int)p.K;
    w.k_at = T::kWgrad ? row - skip : 0;
    w.first = skip / T::kStepK;
    w.f_row = (T::kWgrad ? 0 : lo * p.N) + w.f0;
    w.c_row = (T::kWgrad ? 0 : row) + w.c0;
    w.steps = (int)((uint32_t)(sum + T::kStepK - 1) / T::kStepK);
    const int n = (int)((uint32_t)(sum + T::kStageK - 1) / T::kStageK);
    w.parts = 1;
    w.k0 = 0;
    w.k1 = n;
    if (split > 1) {
      // a part is of whole fetches of scales, and of two stages at least
      const int units = (n + T::kFetch - 1) / T::kFetch;
      w.parts = min(split, max(1, min(n / 2, units)));
      w.k0 = (int)((uint32_t)(units * w.part) / (uint32_t)w.parts) * T::kFetch;
      w.k1 = min(n, (int)((uint32_t)(units * (w.part + 1)) / (uint32_t)w.parts) * T::kFetch);
    }
    return w.part < w.parts && w.cols > 0;
  };
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    return mbar_try(b, parity) || wait_long(b, parity, &s.dead, p.status);
  };
  auto wait_warp = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(kAll, wait(b, parity));
  };

  // A warp's next piece of work, as the copying warp handed it out; false at the end.
  auto take = [&](uint32_t& n, Work& w) -> bool {
    const uint32_t slot = n % kWorks;
    if (!wait_warp(&s.work_full[slot], (n / kWorks) & 1)) return false;
    w = s.work[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.work_free[slot]);
    ++n;
    return w.part >= 0;
  };
  // Given up: copies in flight land before the CTA ends (milliseconds are many times enough).
  auto land = [&]() {
    const long long t0 = clock64();
    while (clock64() - t0 < 20000000) {
    }
  };
  // an arrival at the barrier of the pair's first CTA, which issues the products
  auto arrive_first = [&](uint64_t* b) {
    if constexpr (CG == 2) mbar_arrive_cluster(cluster_addr(b, 0));
    else mbar_arrive(b);
  };

  if (warp < kEpilogueWarps) {
    // ==== results ==============================================================
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t acc_lane = tmem + ((uint32_t)quarter << 21);
    uint32_t taken = 0;
    int done = 0, tiles = 0;
    for (;;) {
      Work w;
      bool go = take(taken, w);
      float* sc = s.scale[tiles++ & 1];
      float gf = 1.0f;
      if (T::kFp4 && go) {
        const SliceScale f = slice_scale(p.f_amax[w.g], p.f_M);
        gf = f.g;
        bool bad = f.bad;
        float gc = 0.0f;
        if (tid < w.cols) {
          const SliceScale c = slice_scale(p.c_amax[p.c_amax_each ? w.c_row + tid : 0], p.c_M);
          gc = c.g;
          bad = bad || c.bad;
        }
        sc[tid] = gc;
        if (bad) flag(p.status, NVFP4_DEV_BAD_AMAX);
      }
      // the columns' scales are there, and the warps go on or end together
      if (!all_of(go)) break;
      const bool sum = w.k1 > w.k0;  // false: a sum over nothing
      const int buf = done & 1;
      if (sum) {
        // (after a timeout the results are not valid, but every barrier is still met)
        wait_warp(&s.acc_full, done & 1);
        fence_after();
      }
      const uint32_t acc = acc_lane + (buf ? kAcc1 : 0);
      const int f = w.f0 + quarter * 32 + lane;
      float* part = p.part + ((int64_t)w.item * CG + rank) * kMatmulPart + quarter * 32 + lane;
      // the results of columns c .. c + n - 1, for the lane's feature
      auto put = [&](int c, auto& v) {
        constexpr int kN = sizeof(v) / sizeof(float);
        if constexpr (T::kFp4) {
#pragma unroll
          for (int i = 0; i < kN; i += 4) {
            const float4 g = *reinterpret_cast<const float4*>(sc + c + i);
            const f2 gff = make_float2(gf, gf);
            const f2 a = f2_mul(f2_mul(make_float2(v[i], v[i + 1]), make_float2(g.x, g.y)), gff);
            const f2 b = f2_mul(f2_mul(make_float2(v[i + 2], v[i + 3]), make_float2(g.z, g.w)), gff);
            v[i] = a.x, v[i + 1] = a.y, v[i + 2] = b.x, v[i + 3] = b.y;
          }
        }
        if (T::kWgrad && p.turn) {
          if constexpr (kN == 32) {
            // a lane's 64 bytes of a row to shared memory, swizzled so that eight rows meet no
            // bank twice, and the warp's box to its place
            if (f - lane >= p.N) return;
            if (lane == 0) bulk_wait_read();  // the last box has left
            __syncwarp();
            uint8_t* at = ring + T::kRing + warp * kTurn;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(at + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]),
                             pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                             pack_bf16x2(v[8 * j + 4], v[8 * j + 5]),
                             pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
            fence_smem_async();
            __syncwarp();
            if (lane == 0) tma_store(&maps.out, w.c0 + c, f, w.g, smem_addr(at));
          } else if (f < p.N) {  // a sum's parts: 16 columns, at 16 bytes (as the map's base)
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                                ((int64_t)w.g * p.N + f) * p.C + w.c0 + c);
#pragma unroll
            for (int j = 0; j < kN / 8; ++j)
              o[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]),
                                pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                                pack_bf16x2(v[8 * j + 4], v[8 * j + 5]),
                                pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
          }
          return;
        }
        const int64_t row0 = T::kWgrad ? (int64_t)w.g * p.C + w.c0 : (int64_t)w.c_row;
        // every lane has a feature, every column is there: no checks
        const bool whole = c + kN <= w.cols && f - lane + 32 <= p.N;
        if (p.out_f32) {
          float* o = static_cast<float*>(p.out) + (row0 + c) * p.N + f;
#pragma unroll
          for (int i = 0; i < kN; ++i, o += p.N)
            if (whole || (c + i < w.cols && f < p.N)) *o = v[i];
        } else if (p.N % 2 == 0) {
          // neighbouring lanes swap, so that each stores two features of one column
          const int odd = lane & 1;
          uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                    (row0 + c + odd) * p.N + (f & ~1));
#pragma unroll
          for (int i = 0; i < kN; i += 2, o += p.N) {
            const uint32_t a = pack_bf16x2(v[i], v[i + 1]), b = __shfl_xor_sync(kAll, a, 1);
            const uint32_t x = __byte_perm(a, b, odd ? 0x3276u : 0x5410u);
            if (whole || (c + i + odd < w.cols && f < p.N)) *o = x;
          }
        } else {
          uint16_t* o = static_cast<uint16_t*>(p.out) + (row0 + c) * p.N + f;
#pragma unroll
          for (int i = 0; i < kN; ++i, o += p.N)
            if (whole || (c + i < w.cols && f < p.N)) *o = (uint16_t)pack_bf16x2(v[i], 0.0f);
        }
      };
      // A warpgroup has every other 32 columns. Those that the two accumulators share come
      // first, and once they are in registers the next tile's products may begin.
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int chunk = 2 * (buf ? i : 3 - i) + half;
        const bool some = chunk * 32 < w.cols;
        uint32_t r[32];
        if (sum && some) {
          tmem_ld32(acc + chunk * 32, r);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0;
        }
        if (i == 0 && sum) {
          // (the reads are complete at tmem_wait_ld, and nothing of memory is handed over: an
          // arrival without cluster scope does for the pair's first CTA as well)
          fence_before();
          __syncwarp();
          if (lane == 0) arrive_first(&s.acc_free);
        }
        if (!some) continue;
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        if (w.parts > 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (chunk * 32 + j < w.cols) part[(chunk * 32 + j) * 128] = v[j];
        } else {
          put(chunk * 32, v);
        }
      }
      if (sum) ++done;
      if (w.parts > 1) {
        // the CTA that takes the tile's last ticket adds the parts in order
        asm volatile("bar.sync 1, %0;" ::"n"(kEpilogueWarps * 32) : "memory");
        if (tid == 0) {
          __threadfence();
          s.last = atomicAdd(&p.tickets[w.tile * CG + rank], 1u) == (uint32_t)w.parts - 1;
          __threadfence();
        }
        asm volatile("bar.sync 1, %0;" ::"n"(kEpilogueWarps * 32) : "memory");
        if (s.last) {
          const float* all =
              p.part + ((int64_t)w.tile * split * CG + rank) * kMatmulPart + quarter * 32 + lane;
#pragma unroll 1
          for (int c = half * 16; c < w.cols; c += 32) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
#pragma unroll 1
            for (int q = 0; q < w.parts; q += 4) {  // loads of four parts in flight
              float r[4][16];
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  r[u][j] = q + u < w.parts && c + j < w.cols
                                ? __ldcg(all + (int64_t)(q + u) * CG * kMatmulPart + (c + j) * 128)
                                : 0.0f;
#pragma unroll
              for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], r[u][j]);
            }
            put(c, v);
          }
          if (tid == 0) p.tickets[w.tile * CG + rank] = 0;
        }
      }
    }
    if (T::kWgrad && lane == 0) bulk_wait_read();
  } else if (warp == kCopyWarp) {
    // ==== codes: one lane to a box; pieces of work for all warps =====================
    Place pl;
    bool ok = true, ended = false;
    int item = pair;
    uint32_t given = 0, at = 0;  // pieces handed out, and which of them is copied now
    // Finding a piece takes some hundred clocks: it is done between copies, while the ring is
    // full, and never by a warp that others wait for.
    auto give = [&](bool now) {
      if (ended || given >= at + kWorks) return;
      const uint32_t slot = given % kWorks, parity = ((given / kWorks) & 1) ^ 1;
      if (now) {
        if (!(ok = wait_warp(&s.work_free[slot], parity))) return;
      } else if (!__all_sync(kAll, mbar_test(&s.work_free[slot], parity))) {
        return;
      }
      Work x;
      for (ended = true; ended && item < items; item += pairs) ended = !work_of(item, x);
      if (ended) x.part = -1;
      if (lane == 0) {
        s.work[slot] = x;
        mbar_arrive(&s.work_full[slot]);
      }
      __syncwarp();
      ++given;
    };
    for (; ok; ++at) {
      if (at == given) give(true);
      if (!ok) break;
      const Work w = s.work[at % kWorks];
      if (w.part < 0) break;
      const int held = ((w.cols + 15) & ~15) / CG;  // columns of this CTA
      const Boxes boxes(held);
      const uint32_t bytes = kFBytes + boxes.rows() * kStageRow;
      const int x0 = w.k_at;
      const int c_row = w.c_row + rank * held + boxes.row(lane);
      const CUtensorMap* c_box = lane < boxes.large ? &maps.c : &maps.c_small;
      for (int k = w.k0; k < w.k1; ++k, pl.next(stages)) {
        const int st = pl.st;
        if (!(ok = wait_warp(&s.empty[st], pl.turn ^ 1))) break;
        const uint32_t dst = smem_addr(ring + st * stage_bytes);
        const uint32_t c_dst = dst + kFBytes + boxes.row(lane) * kStageRow;
        const int x = x0 + k * kStageRow;
        if constexpr (CG == 2) {
          const uint32_t bar = cluster_addr(&s.full[st], 0);
          if (lane == 0) {
            if (rank == 0) mbar_expect(&s.full[st], 2 * bytes);
            tma_load_pair(dst, &maps.f, x, w.f_row, bar);
          }
          __syncwarp();
          if (lane < boxes.count) tma_load_pair(c_dst, c_box, x, c_row, bar);
        } else {
          if (lane == 0) {
            mbar_expect(&s.full[st], bytes);
            tma_load(dst, &maps.f, x, w.f_row, &s.full[st]);
          }
          __syncwarp();
          if (lane < boxes.count) tma_load(c_dst, c_box, x, c_row, &s.full[st]);
        }
        give(false);
      }
    }
    if (!ok) land();
  } else if (warp == kMmaWarp) {
    // ==== products ==============================================================
    uint32_t tiles = 0, taken = 0;
    Place pl;
    bool ok = true;
    Work w;
    while (ok && take(taken, w)) {
      if (rank != 0 || w.k1 <= w.k0) continue;
      const int n16 = (w.cols + 15) & ~15, blocks = (w.cols + 127) >> 7;
      const uint32_t acc = tmem + (tiles & 1 ? kAcc1 : 0);
      if (tiles > 0 && !(ok = wait_warp(&s.acc_free, (tiles - 1) & 1))) break;
      fence_after();
      for (int k = w.k0; k < w.k1; ++k, pl.next(stages)) {
        const int st = pl.st;
        if (!(ok = wait_warp(&s.full[st], pl.turn))) break;
        fence_after();
        if (elect_one()) {
          // (copies to tensor memory and products of one thread run in order: the scales' columns
          // serve every stage)
          const uint32_t at = smem_addr(ring + st * stage_bytes);
          const uint32_t sf = tmem + kScales;
          const uint32_t sf16 = (at + sf_at) >> 4;
          constexpr int kPer = T::kFp4 ? 4 : 1;  // scale columns groups per stage
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            copy_scales<CG>(sf + 4 * j, scale_desc(sf16 + j * 32));
            copy_scales<CG>(sf + 16 + 8 * j, scale_desc(sf16 + T::kSfBlock / 16 + j * 32));
            if (blocks > 1)
              copy_scales<CG>(sf + 16 + 8 * j + 4,
                              scale_desc(sf16 + 2 * T::kSfBlock / 16 + j * 32));
          }
          const uint64_t df = smem_desc(at >> 4, 16), dc = smem_desc((at + kFBytes) >> 4, 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (k * 4 + j >= w.steps) break;
            if (T::kWgrad && k * 4 + j < w.first) continue;
            const bool add = k > w.k0 || j > (T::kWgrad && k == 0 ? w.first : 0);
            if constexpr (T::kFp4)
              mma_nvfp4<CG>(acc, df + 2 * j, dc + 2 * j, nvfp4_mma_desc(CG, n16), sf + 4 * j,
                        sf + 16 + 8 * j, add);
            else
              mma_mxfp8<CG>(acc, df + 2 * j, dc + 2 * j, mxfp8_mma_desc(CG, n16, j), sf, sf + 16,
                            add);
          }
          if constexpr (CG == 2) {
            mma_commit_pair(&s.empty[st]);
            if (k + 1 == w.k1) mma_commit_pair(&s.acc_full);
          } else {
            mma_commit(&s.empty[st]);
            if (k + 1 == w.k1) mma_commit(&s.acc_full);
          }
        }
        __syncwarp();
      }
      ++tiles;
    }
    // nothing is in flight when the tensor memory is freed and the CTAs end
    if (elect_one()) {
      if constexpr (CG == 2) {
        if (rank == 0) mma_commit_pair(&s.end);
      } else {
        mma_commit(&s.end);
      }
      const long long t0 = clock64();
      while (!mbar_try(&s.end, 0) && clock64() - t0 < kWaitCycles) {
      }
    }
    __syncwarp();
  } else if (T::kFp4 && sf_aligned && warp == kScaleWarp) {
    // ==== scales: copies, a lane to 128 rows ======================================
    Place pl;
    bool ok = true;
    uint32_t taken = 0;
    Work w;
    while (ok && take(taken, w)) {
      const Boxes boxes(w.cols);
      const int row = boxes.row(lane - 1), in = lane == 0 ? 0 : 1 + row / 128;  // its 128 rows
      const CUtensorMap* map =
          lane == 0 ? &maps.fs : lane <= boxes.large ? &maps.cs : &maps.cs_small;
      const int y = lane == 0 ? w.f_row : w.c_row + row;
      const uint32_t at = sf_at + (lane == 0 ? 0 : T::kSfBlock + row * T::kStageSf);
      const int held = lane == 0 ? 128 : max(0, min(boxes.rows() - (lane - 1) * 128, 128));
      for (int k = w.k0; k < w.k1; ++k, pl.next(stages)) {
        const int st = pl.st;
        if (!(ok = wait_warp(&s.empty[st], pl.turn ^ 1))) break;
        if (lane <= c_blocks) mbar_expect(&s.raw[lane][st], held * T::kStageSf);
        __syncwarp();
        if (lane <= boxes.count)
          tma_load(smem_addr(ring + st * stage_bytes + at), map, k * T::kStageSf, y,
                   &s.raw[in][st]);
      }
    }
    if (!ok) land();
  } else if (T::kFp4 && warp < kScaleWarp + 3) {
    // ==== scales that are not aligned: copies, a warp to 128 rows ====================
    // The two aligned pieces that hold a stage's 16 bytes of a row, two stages at a time (a
    // warp's copy then finds 32 bytes of 16 rows side by side).
    const int block = warp - kScaleWarp;  // 0 features, 1 and 2 columns
    const uint8_t* base = block == 0 ? p.f_sf : p.c_sf;
    const int64_t rows = block == 0 ? p.f_rows : p.c_rows;
    const uint8_t* end = base + rows * p.sf_stride;
    const int piece = lane & 1;
    Place pl;
    bool ok = true;
    uint32_t taken = 0;
    Work w;
    while (ok && take(taken, w)) {
      if (sf_aligned || block > c_blocks) continue;
      const int64_t row0 = (int64_t)(block == 0 ? w.f_row : w.c_row + 128 * (block - 1)) +
                           (lane >> 1);
      const bool any = block == 0 || 128 * (block - 1) < w.cols;
      for (int k = w.k0; k < w.k1; k += 2) {
        const bool both = k + 1 < w.k1;
        Place next = pl;
        next.next(stages);
        ok = wait_warp(&s.empty[pl.st], pl.turn ^ 1) &&
             (!both || wait_warp(&s.empty[next.st], next.turn ^ 1));
        if (!ok) break;
        if (piece == 0 || both) {
          const int at = (k + piece) * T::kStageSf, valid = min(T::kStageSf, (int)p.sf_stride - at);
          uint8_t* dst = ring + (piece ? next.st : pl.st) * stage_bytes + sf_at +
                         block * T::kSfBlock + (lane >> 1) * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool in = any && row0 + 16 * i < rows;
            const uint8_t* q = in ? base + (row0 + 16 * i) * p.sf_stride + at : base;
            const int off = (int)((uintptr_t)q & 15);
            q -= off;
            // (nothing is read at the array's end or after it)
            const int lo = in ? (int)min((int64_t)16, (int64_t)(end - q)) : 0;
            const int hi =
                in && off + valid > 16 ? (int)min((int64_t)16, (int64_t)(end - q) - 16) : 0;
            cp_async16_zfill(dst + 256 * i, q, lo);
            cp_async16_zfill(dst + (1 + c_blocks) * T::kSfBlock + 256 * i, hi > 0 ? q + 16 : base,
                             hi);
          }
        }
        copies_arrive(&s.raw[block][pl.st]);
        if (both) {
          copies_arrive(&s.raw[block][next.st]);
          pl = next;
        }
        pl.next(stages);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (T::kFp4) {
    // ==== scales: lane l turns rows l, l + 32, l + 64, l + 96 ======================
    const int block = warp - kScaleWarp - 3;
    const uint32_t base = (uint32_t)(uintptr_t)(block == 0 ? p.f_sf : p.c_sf);
    Place pl;
    bool ok = true;
    uint32_t taken = 0;
    Work w;
    while (ok && take(taken, w)) {
      // where a row's bytes begin in its first piece
      const uint32_t row = (uint32_t)(block == 0 ? w.f_row : w.c_row + 128 * (block - 1)) + lane;
      const uint32_t stride = (uint32_t)p.sf_stride, off = base + row * stride;
      for (int k = w.k0; k < w.k1; ++k, pl.next(stages)) {
        const int st = pl.st;
        if (block <= c_blocks) {
          if (!(ok = wait_warp(&s.raw[block][st], pl.turn))) break;
          uint4* at = reinterpret_cast<uint4*>(ring + st * stage_bytes + sf_at +
                                               block * T::kSfBlock) + lane;
          uint4 v[4] = {at[0], at[32], at[64], at[96]};
          if (!sf_aligned) {
            const uint4* hi = at + (1 + c_blocks) * T::kSfBlock / 16;
            const int valid = min(T::kStageSf, (int)p.sf_stride - k * T::kStageSf);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[i] = first_bytes(window16(v[i], hi[32 * i], (off + 32 * i * stride) & 15), valid);
          }
          at[0] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
          at[32] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
          at[64] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
          at[96] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
          fence_smem_async();
        } else if (!(ok = wait_warp(&s.empty[st], pl.turn ^ 1))) {
          break;
        }
        __syncwarp();
        if (lane == 0) arrive_first(&s.full[st]);
      }
    }
  } else if constexpr (!T::kFp4) {
    // ==== MXFP8 scales: two warps to 128 rows =======================================
    // A line of the layout that tensor memory takes holds rows l, l + 32, l + 64 and
    // l + 96; a warp has 16 of the 32 lines. A lane fetches 16 bytes (four stages) of its
    // line's four rows, the lane beside it the next 16, several fetches ahead.
    const int block = (warp - kScaleWarp) >> 1;  // 0 features, 1 and 2 columns
    const int line = ((warp - kScaleWarp) & 1) * 16 + (lane >> 1), piece = lane & 1;
    const uint8_t* base = block == 0 ? p.f_sf : p.c_sf;
    const int64_t rows = block == 0 ? p.f_rows : p.c_rows;
    constexpr int kStages = 2 * T::kFetch;  // of a fetch
    // Where the 16 bytes are aligned they stay as they came; else two aligned pieces are
    // kept and cut at their use.
    auto feed = [&](auto aligned_c, auto ahead_c) {
      constexpr bool kAligned = decltype(aligned_c)::value;
      constexpr int kAhead = decltype(ahead_c)::value;
      const uint8_t* end = base + rows * p.sf_stride;
      const uint32_t row_step = (uint32_t)(32 * p.sf_stride);
      int k = 0;  // the fetch that comes next
      uint32_t taken = 0;
      Work w{};
      bool have = false, ended = false;
      int held = 0;  // fetches that are not stored yet
      uint4 lo[kAhead][4], hi[kAligned ? 1 : kAhead][4];
      uint32_t off[kAhead];            // low bits of the lane's first address
      int count[kAhead], lead[kAhead];  // the end of a fetch's stages (0: none), their begin
      auto fetch = [&](auto slot_c) {
        constexpr int kSlot = decltype(slot_c)::value;
        count[kSlot] = 0;
        while (!have || k >= w.k1) {
          if (ended) return;
          // Work ahead is not waited for while scales are held here: pieces without stages (groups
          // without rows) may fill all that can be handed out until the products of the held
          // scales have run. The slot then stays empty for this turn.
          if (held > 0 && !__all_sync(kAll, mbar_test(&s.work_full[taken % kWorks],
                                                      (taken / kWorks) & 1)))
            return;
          have = take(taken, w);
          if (!have) {
            ended = true;
            return;
          }
          k = w.k0;
          // (a weights' gradient may begin inside 16 aligned bytes)
          if (kAligned && T::kWgrad) k -= (w.k_at / T::kStageK + k) % T::kFetch;
        }
        const int64_t row0 =
            (int64_t)(block == 0 ? w.f_row : w.c_row + 128 * (block - 1)) + line;
        const int at = w.k_at / 32 + k * T::kStageSf + 16 * piece;
        const bool any = (block == 0 || 128 * (block - 1) < w.cols) &&
                         piece * T::kFetch < w.k1 - k;
        const int valid = min((int)p.sf_stride - at, 16);  // bytes of the row in the piece
        count[kSlot] = min(kStages, w.k1 - k);
        ++held;
        lead[kSlot] = max(w.k0 - k, 0);
        k += kStages;
        const uint8_t* first = base + row0 * p.sf_stride + at;
        off[kSlot] = (uint32_t)(uintptr_t)first;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool in = any && row0 + 32 * i < rows;
          const uint8_t* q = first + i * 32 * p.sf_stride;
          const uint4 none = make_uint4(0, 0, 0, 0);
          if constexpr (kAligned) {
            lo[kSlot][i] = in ? __ldg(reinterpret_cast<const uint4*>(q)) : none;
          } else {
            const int o = (int)((uintptr_t)q & 15);
            q -= o;
            lo[kSlot][i] = in ? bytes16(q, end) : none;
            hi[kSlot][i] = in && o + valid > 16 ? bytes16(q + 16, end) : none;
          }
        }
      };
      Place pl;
      // the stages of a fetch, to shared memory; false at the end
      auto store = [&](auto slot_c) -> bool {
        constexpr int kSlot = decltype(slot_c)::value;
        if (count[kSlot] == 0) return !ended || held > 0;
        --held;
        uint32_t x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v = lo[kSlot][i];
          if constexpr (!kAligned)
            v = window16(v, hi[kSlot][i], (off[kSlot] + i * row_step) & 15);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        }
#pragma unroll
        for (int c = 0; c < kStages; ++c) {
          if (c >= count[kSlot]) break;
          if (kAligned && T::kWgrad && c < lead[kSlot]) continue;
          const int st = pl.st;
          if (!wait_warp(&s.empty[st], pl.turn ^ 1)) return false;
          if (block <= c_blocks && piece == c / T::kFetch) {
            uint4* dst = reinterpret_cast<uint4*>(ring + st * stage_bytes + sf_at +
                                                  block * T::kSfBlock) + line;
            constexpr int kLast = T::kFetch - 1;
            *dst = make_uint4(x[0][c & kLast], x[1][c & kLast], x[2][c & kLast], x[3][c & kLast]);
            fence_smem_async();
          }
          __syncwarp();
          if (lane == 0) arrive_first(&s.full[st]);
          pl.next(stages);
        }
        return true;
      };
      ring_of<kAhead>(fetch, store);
    };
    if (sf_aligned)
      feed(std::true_type{}, std::integral_constant<int, 3>{});
    else
      feed(std::false_type{}, std::integral_constant<int, 2>{});
  }
  __syncwarp();
  fence_before();
  if constexpr (CG == 2) {  // nothing of the other CTA's reads or signals here
    cluster_arrive();
    cluster_wait();
  }
  if constexpr (CG == 1) __syncthreads();
  fence_after();
  if (warp == kMmaWarp) {
    if constexpr (CG == 2) tmem_free_pair(tmem, 512);
    else tmem_free(tmem, 512);
  }
}

// Scales in rows of `stride` bytes, copied to rows of `wide` (a multiple of 16), zeros behind a
// row's bytes. A thread to 16 bytes; two arrays, one after the other.
constexpr int kPadThreads = 256;
__global__ void __launch_bounds__(kPadThreads) pad_scales_kernel(
    const uint8_t* a, int64_t a_rows, const uint8_t* b, int64_t b_rows, int stride, int units,
    FastDiv by_units, uint8_t* out) {
  pdl_begin();
  const int64_t n = (a_rows + b_rows) * units;
  for (int64_t i = (int64_t)blockIdx.x * kPadThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kPadThreads) {
    const int64_t row = fastdiv((uint32_t)i, by_units);
    const int at = 16 * (int)(i - row * units), valid = min(16, stride - at);
    const bool first = row < a_rows;
    const uint8_t* base = first ? a : b;
    const uint8_t* end = base + (first ? a_rows : b_rows) * stride;
    const uint8_t* q = base + (first ? row : row - a_rows) * stride + at;
    const uint32_t off = (uint32_t)((uintptr_t)q & 15);
    q -= off;
    const uint4 lo = bytes16(q, end);
    const uint4 hi = off + valid > 16 ? bytes16(q + 16, end) : make_uint4(0, 0, 0, 0);
    reinterpret_cast<uint4*>(out)[i] = first_bytes(window16(lo, hi, off), valid);
  }
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's function that makes tensor maps (the library links the runtime alone).
EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* at = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      at = nullptr;
    return reinterpret_cast<EncodeTiled>(at);
  }();
  return f;
}

// rows x bytes, boxes of box_rows x box_bytes; false if it cannot be made
bool make_map(CUtensorMap* m, const uint8_t* at, int64_t bytes, int64_t rows, int box_bytes,
              int box_rows) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)bytes};
  const cuuint32_t sizes[2] = {(cuuint32_t)box_bytes, (cuuint32_t)box_rows}, steps[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(at), dims, strides, sizes,
           steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
           box_bytes == kStageRow ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// a weights' gradient's bf16 results [E][N][C], boxes of 32 x 32
bool make_out_map(CUtensorMap* m, const MatmulParams& p) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t row = 2 * (cuuint64_t)p.C;
  const cuuint64_t dims[3] = {(cuuint64_t)p.C, (cuuint64_t)p.N, (cuuint64_t)p.E};
  const cuuint64_t strides[2] = {row, row * p.N};
  const cuuint32_t sizes[3] = {32, 32, 1}, steps[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.out, dims, strides, sizes, steps,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, int CG>
cudaError_t launch_t(const MatmulParams& p, const Maps& m, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(matmul_kernel<KIND, CG>, kSmem, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(std::min(sm_count(), kMatmulMaxCtas) & ~(CG - 1)));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kSmem;
  lc.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = CG;
  const int cols = KIND == kMatmulMxWgrad ? p.C : (int)p.c_rows;
  const int c_tiles = (cols + p.c_tile - 1) / p.c_tile;
  MatmulParams q = p;
  q.tiles = c_tiles * ((p.N + kTileF * CG - 1) / (kTileF * CG));
  q.by_tiles = make_fastdiv((uint32_t)std::max(q.tiles, 1));
  int most = (cols + c_tiles - 1) / std::max(c_tiles, 1);
  if (KIND == kMatmulMxWgrad && c_tiles > 1) most = (most + 31) & ~31;
  const int64_t sum = KIND == kMatmulMxWgrad ? p.K / p.E : p.K;
  const int stages = (int)((sum + Kind<KIND>::kStageK - 1) / Kind<KIND>::kStageK);
  const Geometry geo = geometry<KIND, CG>(q.tiles * (KIND == kMatmulMxWgrad ? p.E : 1),
                                          most, stages, (int)lc.gridDim.x / CG,
                                          p.sf_stride % 16 == 0);
  return cudaLaunchKernelEx(&lc, matmul_kernel<KIND, CG>, m, q, geo);
}
// Pairs of CTAs on 256 features by up to 256 columns where there is about one such tile for
// each pair; else single CTAs, with columns that are cut finer while half of the SMs would be
// without work (512 rows, 2048 x 7168: pairs 17.0 us, tiles of 256 columns 18.8, of 128 14.4, of
// 64 13.2; cut finer up to all SMs: 8 x 300 rows, 512 x 512 8.3 us where this takes 7.3).
template <int KIND>
cudaError_t launch_k(MatmulParams p, const Maps& m, cudaStream_t st) {
  constexpr bool kWgrad = KIND == kMatmulMxWgrad;
  const int64_t cols = kWgrad ? p.C : p.c_rows / p.E;  // of a group, on average
  // tiles of c columns in all groups: ragged ones end half a tile early
  auto c_tiles = [&](int64_t c) {
    return kWgrad ? p.E * ((p.C + c - 1) / c)
           : p.E == 1 ? (p.c_rows + c - 1) / c
                      : p.c_rows / c + std::min<int64_t>(p.E, p.c_rows) / 2;
  };
  const int64_t f_tiles = (p.N + kTileF - 1) / kTileF, sms = sm_count();
  auto tile = [&](int c, int shift) {
    p.c_tile = c;
    p.c_shift = shift;
  };
  tile(256, 8);
  if (p.N > kTileF && cols >= kPairCols && (f_tiles + 1) / 2 * c_tiles(256) * 4 >= sms / 2 * 3)
    return launch_t<KIND, 2>(p, m, st);
  if (f_tiles * c_tiles(256) * 2 < sms) tile(128, 7);
  if (f_tiles * c_tiles(128) * 2 < sms) tile(64, 6);
  return launch_t<KIND, 1>(p, m, st);
}

}  // namespace

cudaError_t launch_matmul(int kind, const MatmulParams& given, const uint8_t* f_codes,
                          const uint8_t* c_codes, cudaStream_t st) {
  MatmulParams p = given;
  // Rows of scales that are not whole 16 bytes take the kernel longer, a stage by about kPadGain
  // microseconds; copying them first takes a launch and their bytes twice (8 experts of 1024
  // rows, 2048 x 7136: 114 us as they are, 80 copied first; 5 experts of 140 rows, 1000 x 416
  // in MXFP8: 8.3 and 9.4).
  const int64_t units = (p.sf_stride + 15) / 16, padded = 16 * units;
  if (p.sf_stride % 16 != 0 && (p.f_rows + p.c_rows) * padded <= (int64_t)kMatmulPadBytes) {
    const bool wgrad = kind == kMatmulMxWgrad;
    const int64_t c_tiles = wgrad ? p.E * (((int64_t)p.C + kTileC - 1) / kTileC)
                                  : p.c_rows / kTileC + std::min<int64_t>(p.E, p.c_rows);
    const int64_t stage = kind == kMatmulNvfp4 ? 256 : 128;
    const int64_t stages = c_tiles * ((p.N + kTileF - 1) / kTileF) *
                           (wgrad ? (p.K / p.E + stage - 1) / stage : (p.K + stage - 1) / stage);
    const double here = (double)stages / sm_count() * kPadGain;
    const double copy = 3.0 + 2e-6 * (double)((p.f_rows + p.c_rows) * padded) / 3.0;
    if (here > copy) {
      const int64_t n = (p.f_rows + p.c_rows) * units;
      const int64_t ctas = std::min<int64_t>((n + kPadThreads - 1) / kPadThreads,
                                             (int64_t)sm_count() * 8);
      const cudaError_t e =
          launch_pdl(pad_scales_kernel, dim3((unsigned)ctas), dim3(kPadThreads), st, p.f_sf,
                     p.f_rows, p.c_sf, p.c_rows, (int)p.sf_stride, (int)units,
                     make_fastdiv((uint32_t)units), p.padded);
      if (e != cudaSuccess) return e;
      p.f_sf = p.padded;
      p.c_sf = p.padded + p.f_rows * padded;
      p.sf_stride = padded;
    }
  }
  Maps m{};
  const int64_t bytes = kind == kMatmulNvfp4 ? p.K / 2 : p.K;
  // without rows to sum over no copy is made: a weights' gradient of zeros
  // and where all columns fit half a large box none is used
  const bool large = (kind == kMatmulMxWgrad ? p.C : p.c_rows) > kBox / 2;
  if (bytes > 0 &&
      (!make_map(&m.f, f_codes, bytes, p.f_rows, kStageRow, kTileF) ||
       (large && !make_map(&m.c, c_codes, bytes, p.c_rows, kStageRow, kBox)) ||
       !make_map(&m.c_small, c_codes, bytes, p.c_rows, kStageRow, kBoxSmall)))
    return cudaErrorInvalidValue;
  if (kind == kMatmulNvfp4 && p.sf_stride % 16 == 0 &&
      (!make_map(&m.fs, p.f_sf, p.sf_stride, p.f_rows, 16, kTileF) ||
       (large && !make_map(&m.cs, p.c_sf, p.sf_stride, p.c_rows, 16, kBox)) ||
       !make_map(&m.cs_small, p.c_sf, p.sf_stride, p.c_rows, 16, kBoxSmall)))
    return cudaErrorInvalidValue;
  if (p.turn && !make_out_map(&m.out, p)) return cudaErrorInvalidValue;
  switch (kind) {
    case kMatmulNvfp4: return launch_k<kMatmulNvfp4>(p, m, st);
    case kMatmulMx: return launch_k<kMatmulMx>(p, m, st);
    default: return launch_k<kMatmulMxWgrad>(p, m, st);
  }
}

}  // namespace nvfp4
