// Shared by the int8 kernels and their entry points.
#pragma once
#include "tq4_internal.h"

namespace tq4 {

constexpr int64_t kInt8MaxK = 131072;   // 127 * 127 * k stays below 2^31

enum Int8Mode : int32_t { INT8_DENSE = 0, INT8_UP = 1, INT8_DOWN = 2 };

struct Int8GemmArgs {
  int32_t n, m;             // weight rows (of one expert); dense: tokens
  int32_t row_tiles;        // ceil(n / 128)
  int32_t tok_tiles;        // dense: ceil(m / NT)
  int32_t ksteps;           // ceil(k / 128)
  int32_t mode, dtype;      // Int8Mode; dense: type of y (TQ_DTYPE_*)
  const int4* segs;         // grouped: (expert, first row, rows <= NT, -), else nullptr
  const int32_t* nseg;      // grouped: how many
  const float* xscale;      // [rows of xq]
  const float* wscale;      // [experts][n]
  const int32_t* pairs;     // down: flat slot of each sorted row
  const float* row_w;       // down: router weight of each sorted row
  void* y;                  // dense: y [m][n]; up: h bf16 [rows][n]; down: fp32 [slots][n]
  int32_t test_withhold;    // test hook: a CTA's first tile is never reported (the bounded waits for it run out)
};

// A tensor map over int8 [experts][rows][k] (3-D), or [rows][k] where experts
// is 0 (2-D): box 128 bytes x box_rows, 128-byte swizzle, zeros outside.
bool encode_i8_map(CUtensorMap* m, const int8_t* base, int64_t experts, int64_t rows, int64_t k, int box_rows);

// nt: 16, 32, 64, 128 or 256 tokens a tile (the box rows of tx), or kInt8Pair:
// dense tiles of 256 weight rows (row_tiles counts those) x 256 tokens shared
// by two CTAs (an even grid), whose tx has 128 box rows.
constexpr int kInt8Pair = 512;
cudaError_t launch_int8_gemm(const CUtensorMap& tw, const CUtensorMap& tx, const Int8GemmArgs& a, int nt, int grid,
                             cudaStream_t st);

// Products of at most 16 tokens a tile that quantize their tokens themselves
// (tq4_int8_stream.cu).
constexpr int kStreamTokens = 16;
struct Int8StreamArgs {
  int32_t n, k, m;          // weight rows and columns (of one expert); dense: tokens
  int32_t row_tiles, ksteps;
  int32_t mode, dtype;      // Int8Mode; type of y (dense), TQ_DTYPE_*
  int32_t parts;            // CTAs of a cluster that share a row tile's k (dense; 1: none)
  int32_t topk;             // up: x row of a sorted row = pairs[row] / topk
  int64_t ldx;
  const void* x;            // dense: x; up: x; down: h (bf16, sorted rows)
  const int4* segs;         // grouped: (expert, first row, rows <= 16, -)
  const int32_t* nseg;
  const int32_t* pairs;
  const float* row_w;
  const int32_t* ids;       // grouped without segs: the kernel routes [slots] ids itself,
  const float* topk_w;      // with their weights
  int32_t slots, experts;   // (slots <= kStreamSlots)
  const float* wscale;
  void* y;                  // as Int8GemmArgs
  int32_t test_withhold;    // test hook: a quantizer warp never reports its first codes
};
constexpr int kStreamSlots = 128;
// Whether rows of k elements fit (their codes stay in shared memory).
bool int8_stream_fits(int64_t k);
// The cluster size for a dense product of row_tiles x ksteps.
int int8_stream_parts(int64_t row_tiles, int64_t ksteps, int sms);
cudaError_t launch_int8_stream(int xdtype, const CUtensorMap& tw, const Int8StreamArgs& a, int64_t most_tiles, int sms,
                               cudaStream_t st);

}  // namespace tq4
