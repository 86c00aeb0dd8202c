// matmul.h -- parameter block of the products grouped by expert (matmul.cu),
// between the C ABI (api_linear.cu) and the kernel.
#pragma once
#include <cuda.h>

#include "kv.h"

namespace nvfp4 {

// Rows of output features ("features") and rows that they are multiplied with
// ("columns": tokens, or the other operand's features in a weights' gradient).
struct MatmulParams {
  const uint8_t *f_sf, *c_sf;   // scale bytes of the features' and the columns' rows
  int64_t f_rows, c_rows;       // rows of those matrices
  int64_t sf_stride;            // scale bytes of a row
  int32_t N;                    // features of a group
  int32_t C;                    // weights' gradient: columns of a group
  int64_t K;                    // values of a row (weights' gradient: rows to sum over)
  int32_t E;
  int32_t c_tile, c_shift;      // columns of a tile at most, a power of two, and its logarithm
  int32_t tiles;                // of a group, where that is the same for all (by_tiles divides)
  FastDiv by_tiles;
  const int32_t* start;         // [E + 1], or null: one group of all rows
  const float *c_amax, *f_amax; // NVFP4: outer scales of the columns (one or each) and groups
  int32_t c_amax_each;
  float c_M, f_M;
  void* out;
  int32_t out_f32;
  int32_t turn;                 // weights' gradient: the features are rows of the results, which
                                // leave by tensor map
  uint32_t* tickets;
  float* part;
  uint8_t* padded;              // kMatmulPadBytes
  int32_t* status;
};

enum { kMatmulNvfp4 = 0, kMatmulMx = 1, kMatmulMxWgrad = 2 };

constexpr int kMatmulMaxGroups = 1024;
// The longest sum: one CTA takes at most 2^18 stages of 128 values for a tile, a quarter of a
// second at 1 us each, and the waits' limit is one.
constexpr int64_t kMatmulMaxSum = 1 << 25;
constexpr int kMatmulMaxCtas = 192;
constexpr int kMatmulPart = 256 * 128;  // floats of a partial result
constexpr size_t kMatmulPadBytes = (size_t)64 << 20;  // scales in rows of whole 16 bytes
constexpr size_t kMatmulTicketBytes = (size_t)4 * 2 * kMatmulMaxCtas;
constexpr size_t kMatmulWsBytes =
    kMatmulTicketBytes + (size_t)4 * kMatmulMaxCtas * kMatmulPart + kMatmulPadBytes;

cudaError_t launch_matmul(int kind, const MatmulParams& p, const uint8_t* f_codes,
                          const uint8_t* c_codes, cudaStream_t st);

}  // namespace nvfp4
