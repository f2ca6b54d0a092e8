// The int8 tensor-core product: acc[t][n] = sum_k xq[t][k] wq[n][k] (exact
// int32 sums), then v = (fp32(acc) sx[t]) sw[n] and one of three epilogues.
//
// The weight is the M operand (128 rows of W, one per tensor-memory lane) and
// NT tokens are the N operand, so that one kernel serves a single token and a
// long prompt: only NT changes, and any n, odd ones too, ends in plain stores.
// Grouped launches (the experts of a MoE) walk the segments -- at most NT
// consecutive rows of one expert -- that the routing kernel wrote.
//   warp 0     TMA producer: 128 x 128 B of W and NT x 128 B of xq a stage;
//   warp 1     one thread issues tcgen05.mma kind::i8 (K = 32), 4 a stage,
//              into one of two tensor-memory accumulators;
//   warp 2     allocates / frees tensor memory;
//   warps 4-   epilogue, thread = weight row; of tiles of 64 tokens or more
//              two warps share 32 rows, each with half of the tokens (one warp
//              per scheduler is bound by latency: the down projection of 4096
//              tokens x 6 of 128 experts took 262 us).
// A tile that holds fewer than NT tokens multiplies only those, rounded up to 16.
// Bound, in the grouped launches of 4096 tokens x 6 of 128 experts, by DRAM (up
// 135 us for 795 MB, down 165 us for 947 MB: 5.9 and 5.7 TB/s); in dense ones
// of one wave by the latency of a k step, 0.23 us (512 x 4096 x 4096 13.5 us).
// A tile's k is never cut between CTAs: with the parts left in memory and
// summed by the CTA that ends last, 4096 x 4096 took 20 to 28 us at 32 to 128
// tokens, against 15 us for half or a quarter as many CTAs with whole tiles.
#include "tq4_int8_mma.cuh"

namespace tq4 {
namespace {

constexpr int kRows = 128;       // weight rows of a tile
constexpr int kStep = 128;       // bytes of k per stage
constexpr int kABytes = kRows * kStep;

template <int NT>
struct Shape {
  static constexpr int kStageBytes = kABytes + NT * kStep;
  static constexpr int kStages = (200 * 1024) / kStageBytes;
  static constexpr int kTmemCols = 2 * NT < 32 ? 32 : 2 * NT;
  static constexpr int kParts = NT >= 64 ? 2 : 1;   // warps that share 32 rows in the epilogue
  static constexpr int kEpilogue = 128 * kParts;    // its threads
  static constexpr int kThreads = 128 + kEpilogue;
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStageBytes + 1024;
};

template <int NT>
struct Shared {
  uint64_t full[Shape<NT>::kStages];
  uint64_t empty[Shape<NT>::kStages];
  uint64_t dfull[2];
  uint64_t dempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int filled;                                       // copies sent to the ring
  int epi_ok[2];
  alignas(16) float sx[2][NT < 32 ? 32 : NT];       // the tile's token scales,
  alignas(16) float tw[2][NT < 32 ? 32 : NT];       // router weights and
  alignas(16) int32_t slot[2][NT < 32 ? 32 : NT];   // slots (down only)
};

// Where a tile lies: expert, first row of W, first token row and how many.
struct Place {
  int32_t expert, row0, tok0, ntok;
};
template <int NT, bool GROUPED>
__device__ __forceinline__ Place place_of(const Int8GemmArgs& a, int32_t tile) {
  Place p;
  if (GROUPED) {
    const int32_t s = tile / a.row_tiles;
    const int4 sg = __ldcg(a.segs + s);
    p.expert = sg.x;
    p.row0 = (tile - s * a.row_tiles) * kRows;
    p.tok0 = sg.y;
    p.ntok = sg.z;
  } else {
    const int32_t r = tile / a.tok_tiles;
    p.expert = 0;
    p.row0 = r * kRows;
    p.tok0 = (tile - r * a.tok_tiles) * NT;
    p.ntok = min(NT, a.m - p.tok0);
  }
  return p;
}

// The 32 tokens (columns c0.. of the tile) of one weight row, from their sums.
// Scales come from shared memory: a global load between the stores would wait
// for its latency 32 times over (the compiler cannot move it past a store).
__device__ __forceinline__ void scale32(const float* sx, float sw, const int32_t (&acc)[32], float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    const float4 s = *reinterpret_cast<const float4*>(sx + j);
    v[j] = __fmul_rn(__fmul_rn(static_cast<float>(acc[j]), s.x), sw);
    v[j + 1] = __fmul_rn(__fmul_rn(static_cast<float>(acc[j + 1]), s.y), sw);
    v[j + 2] = __fmul_rn(__fmul_rn(static_cast<float>(acc[j + 2]), s.z), sw);
    v[j + 3] = __fmul_rn(__fmul_rn(static_cast<float>(acc[j + 3]), s.w), sw);
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 16-bit rows y[token][n] from 32 tokens of one weight row per lane.  Where n
// is even, lanes pair up: of two tokens the even lane takes the first and the
// odd lane the second, for both rows, so that each store is 4 bytes.
template <bool BF16>
__device__ __forceinline__ void store16(uint16_t* y, int64_t n, int row, int rows_left, bool pairs, int ntok,
                                        const float (&v)[32]) {
  if (pairs) {
    const bool odd = row & 1;
    uint32_t* at = reinterpret_cast<uint32_t*>(y + (odd ? n : 0) + (row & ~1));
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
      const uint32_t w = odd ? pack16<BF16>(other, v[j + 1]) : pack16<BF16>(v[j], other);
      if (rows_left > 0 && j + (odd ? 1 : 0) < ntok) at[j * (n >> 1)] = w;
    }
  } else if (rows_left > 0) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < ntok) y[j * n + row] = static_cast<uint16_t>(pack16<BF16>(v[j], 0.0f));
  }
}

// A thread's share of a tile: one weight row, tokens [col0, col0 + cols).
template <int NT, bool GROUPED>
__device__ __forceinline__ void finish_columns(const Int8GemmArgs& a, const Place& pl, int row, float sw,
                                               uint32_t d_addr, int col0, int cols, const float* sx, const float* tw,
                                               const int32_t* slot) {
#pragma unroll 1
  for (int c = col0; c < min(pl.ntok, col0 + cols); c += 32) {
    int32_t acc[32];
    {
      uint32_t r0[16], r1[16];
      tmem_ld16(d_addr + c, r0);
      if (NT > 16) tmem_ld16(d_addr + c + 16, r1);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        acc[j] = static_cast<int32_t>(r0[j]);
        acc[16 + j] = NT > 16 ? static_cast<int32_t>(r1[j]) : 0;
      }
    }
    float v[32];
    scale32(sx + c, sw, acc, v);
    const int left = pl.ntok - c;
    const int64_t tok = pl.tok0 + c;
    if (GROUPED && a.mode == INT8_DOWN) {
      float* z = static_cast<float*>(a.y) + row;
      if (row < a.n)
#pragma unroll
        for (int j = 0; j < (NT < 32 ? NT : 32); ++j)
          if (j < left) z[static_cast<int64_t>(slot[c + j]) * a.n] = __fmul_rn(v[j], tw[c + j]);
    } else if (!GROUPED && a.dtype == TQ_DTYPE_F32) {
      float* y = static_cast<float*>(a.y) + tok * a.n + row;
      if (row < a.n)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j < left) y[static_cast<int64_t>(j) * a.n] = v[j];
    } else {
      if (GROUPED) {   // up
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float r = v[j] < 0.0f ? 0.0f : v[j];   // (a NaN stays)
          v[j] = __fmul_rn(r, r);
        }
      }
      uint16_t* y = static_cast<uint16_t*>(a.y) + tok * a.n;
      const bool pairs = (a.n & 1) == 0;
      if (!GROUPED && a.dtype == TQ_DTYPE_F16) store16<false>(y, a.n, row, a.n - row, pairs, left, v);
      else store16<true>(y, a.n, row, a.n - row, pairs, left, v);
    }
  }
}

// (A kernel for dense and one for grouped launches: code that is not there need
// not be fetched.)
template <int NT, bool GROUPED>
__global__ void __launch_bounds__(Shape<NT>::kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ Int8GemmArgs a) {
  using S = Shape<NT>;
  __shared__ Shared<NT> sh;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], S::kEpilogue);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 2) {
    tmem_alloc(&sh.tmem_base, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = sh.tmem_base;
  volatile int* abortp = &sh.abort_flag;
  // A grouped launch learns its segments from the kernels before it.  A dense
  // one knows its tiles and reads only the weight (which no kernel of this
  // call writes) before its producer waits for the quantized activations.
  if (GROUPED) pdl_wait();
  const int32_t tiles = GROUPED ? __ldcg(a.nseg) * a.row_tiles : a.row_tiles * a.tok_tiles;
  // In grouped launches every role learns the place of its next tile (and the
  // epilogue that tile's scales) while it works on one: these loads' latencies
  // were most of a tile of few k steps (620 rows x 1888 x 224 of 30 experts:
  // 11.5 us, 14.8 without).
  auto place_at = [&](int tile) {
    Place p{};
    if (tile < tiles) p = place_of<NT, GROUPED>(a, tile);
    return p;
  };
  Place next{};
  if (GROUPED) next = place_at(blockIdx.x);
  auto step = [&](int tile) {   // this tile's place, and the next one's on its way
    if (!GROUPED) return place_of<NT, GROUPED>(a, tile);
    const Place p = next;
    next = place_at(tile + gridDim.x);
    return p;
  };

  if (warp == 0) {
    if (lane == 0) {
      int early = 0;   // stages whose weight half is already on its way
      if (!GROUPED) {
        for (int tile = blockIdx.x; tile < tiles && early < S::kStages; tile += gridDim.x) {
          const Place pl = place_of<NT, GROUPED>(a, tile);
          for (int kk = 0; kk < a.ksteps && early < S::kStages; ++kk, ++early) {
            mbar_arrive_expect_tx(&sh.full[early], S::kStageBytes);
            tma_load_3d(smem + early * S::kStageBytes, &tm_w, &sh.full[early], kk * kStep, pl.row0, pl.expert);
          }
        }
        pdl_wait();
      }
      int li = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
        const Place pl = step(tile);
        for (int kk = 0; kk < a.ksteps; ++kk, ++li) {
          uint8_t* st = smem + s * S::kStageBytes;
          if (li >= early) {
            if (!mbar_wait(&sh.empty[s], ph ^ 1u, abortp)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sh.full[s], S::kStageBytes);
            tma_load_3d(st, &tm_w, &sh.full[s], kk * kStep, pl.row0, pl.expert);
          }
          tma_load_2d(st + kABytes, &tm_x, &sh.full[s], kk * kStep, pl.tok0);
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      sh.filled = li;
    }
  } else if (warp == 1) {
    // The whole warp walks, one elected lane issues: values that are the same
    // in every lane stay in the uniform registers that the MMA takes them
    // from.
    int s = 0, ti = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < tiles; tile += gridDim.x) {
      const int db = ti & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sh.dempty[db], ((ti >> 1) & 1) ^ 1u, abortp))) break;
      tc_fence_after();
      const uint32_t d_addr = tmem + db * NT;
      const uint32_t idesc = idesc_i8(kRows, (step(tile).ntok + 15) & ~15);
      for (int kk = 0; kk < a.ksteps; ++kk) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], ph, abortp));
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = sdesc_k128(smem_u32(smem + s * S::kStageBytes));
        const uint64_t bd = sdesc_k128(smem_u32(smem + s * S::kStageBytes + kABytes));
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kStep / 32; ++q)
            mma_i8(d_addr, ad + q * 2, bd + q * 2, idesc, (kk | q) ? 1u : 0u);   // (32 bytes on: 2 units of 16)
          mma_commit(&sh.empty[s]);
        }
        __syncwarp();
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (ok && !(a.test_withhold && ti == 0) && elect_one()) mma_commit(&sh.dfull[db]);
      __syncwarp();
      ++ti;
    }
    if (elect_one()) {
      mma_commit(&sh.mma_done);
      int8_drain_wait(&sh.mma_done, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    pdl_wait();   // the scales come from the kernel before
    const int t = (warp & 3) * 32 + lane;       // the weight row,
    const int part = (warp - 4) >> 2;           // and which of its tokens:
    constexpr int kCols = NT / S::kParts;
    const int col0 = part * kCols;              // columns [col0, col0 + kCols)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int j = part * 128 + t;               // (and whose scale it fetches)
    float sx = 0.0f, tw = 0.0f, sw = 0.0f;      // of the next tile
    int32_t slot = 0;
    auto fetch = [&](const Place& p) {
      const bool in = j < p.ntok;
      sx = in ? __ldcg(a.xscale + p.tok0 + j) : 0.0f;
      if (GROUPED && a.mode == INT8_DOWN) {
        slot = in ? __ldcg(a.pairs + p.tok0 + j) : 0;
        tw = in ? __ldcg(a.row_w + p.tok0 + j) : 0.0f;
      }
      sw = p.ntok > 0 && p.row0 + t < a.n ? __ldcg(a.wscale + static_cast<int64_t>(p.expert) * a.n + p.row0 + t) : 0.0f;
    };
    Place pl = next;
    if (GROUPED) {
      fetch(pl);
      next = place_at(blockIdx.x + gridDim.x);
    }
    int ti = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++ti) {
      const int db = ti & 1;
      if (!GROUPED) {
        pl = place_of<NT, GROUPED>(a, tile);
        fetch(pl);
      }
      // (the buffers of the last tile but one: every thread has left it)
      if (j < NT) {
        sh.sx[db][j] = sx;
        if (GROUPED && a.mode == INT8_DOWN) {
          sh.slot[db][j] = slot;
          sh.tw[db][j] = tw;
        }
      }
      const float sw_here = sw;
      const Place here = pl;
      if (GROUPED) {
        fetch(next);
        pl = next;
        next = place_at(tile + 2 * gridDim.x);
      }
      if (t == 0 && part == 0) sh.epi_ok[db] = mbar_wait(&sh.dfull[db], (ti >> 1) & 1, abortp) ? 1 : 0;
      named_bar_sync(1, S::kEpilogue);
      if (!sh.epi_ok[db]) break;
      tc_fence_after();
      finish_columns<NT, GROUPED>(a, here, here.row0 + t, sw_here, tmem + lane_base + db * NT, col0, kCols, sh.sx[db],
                                  sh.tw[db], sh.slot[db]);
      tc_fence_before();
      mbar_arrive(&sh.dempty[db]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, S::kTmemCols);
  // Where a wait ran out, copies may be in flight.  (Not before here: a role
  // may give up after the last copy was sent.)
  if (threadIdx.x == 0 && *abortp) int8_land_copies(sh.full, S::kStages, sh.filled);
}

// ------------------------------------------------------------------ pairs
// The product of many tokens: two CTAs (a cluster) share a tile of 256 weight
// rows x 256 tokens.  Each copies its own 128 rows of W and half of the
// tokens, 32 KB a k step instead of 48 KB for half a tile, and the MMAs of
// cta_group::2, issued by the first CTA, read both halves; each CTA finishes
// its own 128 rows.  The first CTA's `full` barriers count the bytes of both,
// its commits free the stages of both, and its `dempty` counts the epilogue
// warps of both.  Bound by the tensor cores: 8192 x 14336 x 4096 in 286 us, 3.4
// POP/s, as a burst; 335 to 360 us under the power limit.  (Alone, a CTA's 48 KB a k
// step took 324 and 385 us.)  The MMAs' last arrival goes to both CTAs, so the
// second waits for its own too before it leaves.
constexpr int kPairTok = 256;
constexpr int kPairStageBytes = kABytes + kPairTok / 2 * kStep;
constexpr int kPairStages = (200 * 1024) / kPairStageBytes;
constexpr int kPairThreads = 384, kPairEpilogue = 256;
constexpr size_t kPairSmem = static_cast<size_t>(kPairStages) * kPairStageBytes + 1024;

struct PairShared {
  uint64_t full[kPairStages];
  uint64_t empty[kPairStages];
  uint64_t dfull[2];
  uint64_t dempty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int filled[2];                 // stages that each CTA's copies were sent to (the first CTA's memory)
  int gave_up;                   // in either CTA
  int epi_ok[2];
  alignas(16) float sx[2][kPairTok];
};

// Rows of the pair's tile: the tokens are cut in two halves of `half`.
__device__ __forceinline__ Place place_of_pair(const Int8GemmArgs& a, int32_t tile, int rank, int& half) {
  Place p;
  const int32_t r = tile / a.tok_tiles;
  p.expert = 0;
  p.row0 = r * (2 * kRows) + rank * kRows;
  p.tok0 = (tile - r * a.tok_tiles) * kPairTok;
  p.ntok = min(kPairTok, a.m - p.tok0);
  half = (p.ntok + 31) / 32 * 16;
  return p;
}

// Where a wait ran out: waits for both CTAs' copies in flight, whose bytes the
// first CTA's barriers count.  One of the two may have sent more.
__device__ __noinline__ void land_pair(PairShared& sh) {
  const int own = sh.filled[0], other = sh.filled[1], most = max(own, other);
  for (int i = max(0, most - kPairStages); i < most; ++i) {
    uint64_t* bar = &sh.full[i % kPairStages];
    if (i >= own) mbar_arrive_expect_tx(bar, kPairStageBytes);   // the second CTA's alone
    else if (i >= other) mbar_complete_tx(bar, kPairStageBytes);
    int8_drain_wait(bar, (i / kPairStages) & 1);
  }
}

__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
    int8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ Int8GemmArgs a) {
  __shared__ PairShared sh;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.dfull[i], 1);
      mbar_init(&sh.dempty[i], 2 * kPairEpilogue / 32);
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort_flag = sh.gave_up = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  if (warp == 2) {
    tmem_alloc2(&sh.tmem_base, 512);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();   // both CTAs' barriers are there
  cluster_wait();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = sh.tmem_base;
  volatile int* abortp = &sh.abort_flag;
  const int tiles = a.row_tiles * a.tok_tiles, tile0 = blockIdx.x / 2, stride = gridDim.x / 2;

  if (warp == 0) {
    if (lane == 0) {
      int early = 0;   // stages whose weight half is already on its way
      for (int tile = tile0; tile < tiles && early < kPairStages; tile += stride) {
        int half;
        const Place pl = place_of_pair(a, tile, rank, half);
        for (int kk = 0; kk < a.ksteps && early < kPairStages; ++kk, ++early) {
          if (rank == 0) mbar_arrive_expect_tx(&sh.full[early], 2 * kPairStageBytes);
          tma_load_3d_pair(smem + early * kPairStageBytes, &tm_w, in_cta(&sh.full[early], 0), kk * kStep, pl.row0, 0);
        }
      }
      pdl_wait();
      int li = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < tiles; tile += stride) {
        int half;
        const Place pl = place_of_pair(a, tile, rank, half);
        for (int kk = 0; kk < a.ksteps; ++kk, ++li) {
          uint8_t* st = smem + s * kPairStageBytes;
          const uint32_t bar = in_cta(&sh.full[s], 0);
          if (li >= early) {
            if (!mbar_wait(&sh.empty[s], ph ^ 1u, abortp)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * kPairStageBytes);
            tma_load_3d_pair(st, &tm_w, bar, kk * kStep, pl.row0, 0);
          }
          tma_load_2d_pair(st + kABytes, &tm_x, bar, kk * kStep, pl.tok0 + rank * half);
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      store_remote(in_cta(&sh.filled[rank], 0), li);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, ti = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; ok && tile < tiles; tile += stride, ++ti) {
        const int db = ti & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&sh.dempty[db], ((ti >> 1) & 1) ^ 1u, abortp))) break;
        tc_fence_after();
        int half;
        place_of_pair(a, tile, rank, half);
        const uint32_t d_addr = tmem + db * kPairTok, idesc = idesc_i8(2 * kRows, 2 * half);
        for (int kk = 0; kk < a.ksteps; ++kk) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sh.full[s], ph, abortp));
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sdesc_k128(smem_u32(smem + s * kPairStageBytes));
          const uint64_t bd = sdesc_k128(smem_u32(smem + s * kPairStageBytes + kABytes));
          if (elect_one()) {
#pragma unroll
            for (int q = 0; q < kStep / 32; ++q)   // (32 bytes on: 2 units of 16)
              mma_i8_pair(d_addr, ad + q * 2, bd + q * 2, idesc, (kk | q) ? 1u : 0u);
            mma_commit_pair(&sh.empty[s]);
          }
          __syncwarp();
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok && !(a.test_withhold && ti == 0) && elect_one()) mma_commit_pair(&sh.dfull[db]);
        __syncwarp();
      }
      if (elect_one()) {
        mma_commit_pair(&sh.mma_done);
        int8_drain_wait(&sh.mma_done, 0);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    pdl_wait();   // the scales come from the kernel before
    const int t = (warp & 3) * 32 + lane;
    const int col0 = ((warp - 4) >> 2) * (kPairTok / 2);   // two warps share 32 rows, half of the tokens each
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int ti = 0;
    for (int tile = tile0; tile < tiles; tile += stride, ++ti) {
      const int db = ti & 1;
      int half;
      const Place pl = place_of_pair(a, tile, rank, half);
      {
        const int j = threadIdx.x - 128;   // (the buffer of the last tile but one: every thread has left it)
        sh.sx[db][j] = j < pl.ntok ? __ldcg(a.xscale + pl.tok0 + j) : 0.0f;
      }
      if (threadIdx.x == 128) sh.epi_ok[db] = mbar_wait(&sh.dfull[db], (ti >> 1) & 1, abortp) ? 1 : 0;
      named_bar_sync(1, kPairEpilogue);
      if (!sh.epi_ok[db]) break;
      tc_fence_after();
      const int row = pl.row0 + t;
      const float sw = row < a.n ? __ldcg(a.wscale + row) : 0.0f;
      finish_columns<kPairTok, false>(a, pl, row, sw, tmem + lane_base + db * kPairTok, col0, kPairTok / 2, sh.sx[db],
                               nullptr, nullptr);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(in_cta(&sh.dempty[db], 0));
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abortp)
    for (int i = 0; i < 2; ++i) store_remote(in_cta(&sh.gave_up, i), 1);
  cluster_arrive();   // neither CTA leaves, or frees its tensor memory, while the other may still reach it
  cluster_wait();
  tc_fence_after();
  if (sh.gave_up) {   // (the same in both)
    if (rank == 0 && threadIdx.x == 0) land_pair(sh);
    cluster_arrive();
    cluster_wait();
  }
  // The MMAs' last arrivals are sent to both CTAs.  The first has seen its own.
  if (rank == 1 && threadIdx.x == 0) int8_drain_wait(&sh.mma_done, 0);
  if (warp == 2) tmem_dealloc2(tmem, 512);
}

cudaError_t launch_pair(const CUtensorMap& tw, const CUtensorMap& tx, const Int8GemmArgs& a, int grid,
                        cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(int8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(kPairSmem));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, int8_pair_kernel, tw, tx, a);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

template <int NT, bool GROUPED>
cudaError_t launch_as(const CUtensorMap& tw, const CUtensorMap& tx, const Int8GemmArgs& a, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(int8_gemm_kernel<NT, GROUPED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(Shape<NT>::kSmem));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(Shape<NT>::kThreads);
  cfg.dynamicSmemBytes = Shape<NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, int8_gemm_kernel<NT, GROUPED>, tw, tx, a);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}
template <int NT>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const Int8GemmArgs& a, int grid, cudaStream_t st) {
  return a.segs ? launch_as<NT, true>(tw, tx, a, grid, st) : launch_as<NT, false>(tw, tx, a, grid, st);
}

}  // namespace

cudaError_t launch_int8_gemm(const CUtensorMap& tw, const CUtensorMap& tx, const Int8GemmArgs& a, int nt, int grid,
                             cudaStream_t st) {
  switch (nt) {
    case kInt8Pair: return launch_pair(tw, tx, a, grid, st);
    case 16: return launch<16>(tw, tx, a, grid, st);
    case 32: return launch_as<32, false>(tw, tx, a, grid, st);   // (segments have 16, 64, 128 or 256 rows)
    case 64: return launch<64>(tw, tx, a, grid, st);
    case 128: return launch<128>(tw, tx, a, grid, st);
    default: return launch<256>(tw, tx, a, grid, st);
  }
}

}  // namespace tq4
