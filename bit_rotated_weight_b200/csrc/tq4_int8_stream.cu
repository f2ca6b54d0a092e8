// The int8 product for few tokens (at most 16 a tile): one pass over the
// weight, which is all the time there is; the tokens are quantized in the same
// kernel, while the weight's first tiles are on their way.
//
// Row tiles of 128 weight rows are the M operand of tcgen05.mma kind::i8, the
// tile's tokens the N operand.
//   warp 0      TMA producer of the weight, 16 KB a stage;
//   warps 1-3   one thread each issues the MMAs of every third stage into its
//               own accumulator (one thread takes about 360 ns a stage, less
//               than 50 GB/s of weight; the integer sums may be split at will).
//               Where stages are used again their number is a multiple of
//               three, so that a stage is always the same thread's: a thread
//               that waited for another's stage could be a whole turn ahead of
//               its barrier, and a parity says nothing about two turns;
//   warps 4-7   epilogue, thread = weight row;
//   warps 8-15  quantize the tokens into the MMAs' B tiles (128-byte swizzle):
//               rows' largest values, then codes, 16 of them a thread a turn.
// Persistent form: a CTA takes a contiguous range of (segment, row tile), so
// that a segment's tokens are quantized about once per CTA.  (Their codes have
// one buffer: a second one took the room of three weight stages, and an SM's
// rate is its stages over the 2 us from a stage's copy to its release; 1 token
// of 6 x 128 experts 20.1 us, 21.3 with two.)
// Cluster form, for a dense product of few row tiles: `parts` CTAs share a row
// tile, each with a range of k.  They exchange the rows' largest values and
// their int32 sums by asynchronous stores into each other's shared memory that
// the receiver counts in bytes: no workspace, no second kernel.
// Grouped, with at most 128 slots, every CTA sorts the slots by expert itself
// (a count of smaller ids per slot, 0.5 to 1 us): a kernel for that took 3 us of
// a token's 24, and its results came three memory latencies later.  The down projection
// does so, and starts its weight copies, before it waits for the up projection.
// Role loops are not unrolled: a call of a few microseconds runs most of the
// code once, and fetching instructions was most of its time.
// Every wait on an mbarrier is bounded.  Where one runs out its CTA stores
// nothing more and leaves when nothing is on its way to it: its own copies, and
// what the other CTAs of a cluster send, who all end together (0.08 us of 8.9).
//
// Measured: 16 x 4096 x 4096 8.9 us a call in a graph, 1 x 4096 x 2688 6.8 us
// (17 and 11 MB: 2.6 and 1.7 us of DRAM), a chain of latencies: the launch 2,
// the tokens' loads 1.2, their maxima across the cluster 1, codes 0.5 to 1, the
// MMAs 0.8, the exchange of sums 0.7.  The two projections of 16 tokens x 6 of
// 128 experts (686 MB) 110 to 116 us, 5.9 to 6.2 TB/s, DRAM; those of one token (60 MB)
// 15 us, 90 and 126 tiles for 148 SMs at 41 GB/s each.
#include "tq4_int8_mma.cuh"
#include "tq4_int8_rows.cuh"

namespace tq4 {
namespace {

constexpr int kRows = 128, kStep = 128, kStageBytes = kRows * kStep;
constexpr int kTok = kStreamTokens;
constexpr int kTileB = kTok * kStep;       // bytes of a k step's B tile
constexpr int kThreads = 512, kQuantThreads = 256, kEpilogue = 128;
constexpr int kIssuers = 3;
constexpr int kAcc = 64;                   // tensor-memory columns between the two sets of accumulators
constexpr int kMaxStages = 12;
constexpr int kSpace = 208 * 1024;         // the tokens' codes and the weight stages
constexpr int kHold = 4;                   // turns whose values a quantizer thread keeps between its two passes
constexpr int kPartRow = 20;               // ints of a row's partial sums (16, and padding against bank conflicts)
constexpr int kMaxParts = 8;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t dfull[2], dempty[2];
  uint64_t bfull, bempty;
  uint64_t drained[kIssuers];
  uint64_t maxima, sums;                   // cluster form: what the other CTAs send has arrived
  uint32_t tmem_base;
  int abort_flag;
  int filled;                              // copies sent to the ring
  int quit;                                // a quantizer's wait ran out
  uint32_t top[kTok];                      // largest |x| of each token, as bits (persistent form)
  uint32_t tops[kMaxParts][kTok];          // [CTA][row, or warp of a row] (cluster form)
  float sx[kTok], tw[kTok];
  int32_t slot[kTok];
  alignas(16) int32_t part[kRows * kPartRow];   // cluster form: [CTA][its rows][token]
  // routing in the kernel
  int32_t nseg;
  alignas(16) int32_t id[kStreamSlots];
  alignas(16) int32_t sub[kStreamSlots];   // segments of a slot's expert, at its first slot
  int4 segs[kStreamSlots];
  int32_t pairs[kStreamSlots];
  float row_w[kStreamSlots];
};

// Sorts the slots by expert, by the whole block: a slot's row is the number of
// slots with a smaller id, or the same id earlier.  Four threads count for a
// slot (one each took 10 us of a layer with 128 slots).  Ids out of range are
// left out.  (The ids are ready before this call's first kernel.)
__device__ __forceinline__ void route(Shared& sh, const Int8StreamArgs& a) {
  static_assert(kThreads == 4 * kStreamSlots, "four threads a slot");
  const int t = threadIdx.x >> 2, part = threadIdx.x & 3;
  if (threadIdx.x == 0) sh.nseg = 0;
  int32_t id = INT32_MAX;
  float w = 0.0f;
  if (t < a.slots) {
    id = __ldcg(a.ids + t);
    w = __ldcg(a.topk_w + t);
    if (id < 0 || id >= a.experts) {
      if (blockIdx.x == 0 && part == 0) raise_status(TQ_DEV_BAD_ROUTING);
      id = INT32_MAX;
    }
  }
  if (part == 0) {
    sh.id[t] = id;
    sh.sub[t] = 0;
  }
  __syncthreads();
  auto all = [](int v) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
    return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
  };
  int less = 0, same = 0, before = 0;
#pragma unroll 1
  for (int q = 4 * part; q < a.slots; q += 16) {
    const int4 o = *reinterpret_cast<const int4*>(&sh.id[q]);
    less += (o.x < id) + (o.y < id) + (o.z < id) + (o.w < id);
    same += (o.x == id) + (o.y == id) + (o.z == id) + (o.w == id);
    before += (o.x == id && q < t) + (o.y == id && q + 1 < t) + (o.z == id && q + 2 < t) + (o.w == id && q + 3 < t);
  }
  less = all(less), same = all(same), before = all(before);
  const bool valid = id != INT32_MAX;
  if (valid && part == 0) {
    sh.pairs[less + before] = t;
    sh.row_w[less + before] = w;
    if (before == 0) sh.sub[t] = (same + kTok - 1) / kTok;
  }
  __syncthreads();
  int at = 0;   // segments of smaller ids
#pragma unroll 1
  for (int q = 4 * part; q < a.slots; q += 16) {
    const int4 o = *reinterpret_cast<const int4*>(&sh.id[q]), n = *reinterpret_cast<const int4*>(&sh.sub[q]);
    at += (o.x < id ? n.x : 0) + (o.y < id ? n.y : 0) + (o.z < id ? n.z : 0) + (o.w < id ? n.w : 0);
  }
  at = all(at);
  if (valid && before == 0 && part == 0) {
    for (int i = 0; i < same; i += kTok) sh.segs[at++] = make_int4(id, less + i, min(kTok, same - i), 0);
    atomicAdd(&sh.nseg, (same + kTok - 1) / kTok);
  }
  __syncthreads();
}

// Quantizer threads of a row, for a tile of `tokens` rows.
__device__ __forceinline__ int threads_per_row(int tokens) {
  int t = kQuantThreads;
  while (t * tokens > kQuantThreads) t >>= 1;
  return t;
}

// 16 values of a row, as loaded.
template <typename T>
struct Sixteen {
  static constexpr int kVecs = 16 / Vec<T>::N;
  uint4 raw[kVecs];
  // `wide`: rows lie on 16-byte boundaries
  __device__ __forceinline__ void load(const T* at, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) raw[i] = __ldcg(reinterpret_cast<const uint4*>(at) + i);
    } else {
      load_narrow(at);
    }
  }
  __device__ __noinline__ void load_narrow(const T* at) {
    alignas(16) T v[16];
    for (int i = 0; i < 16; ++i) v[i] = at[i];
    for (int i = 0; i < kVecs; ++i) raw[i] = reinterpret_cast<const uint4*>(v)[i];
  }
  __device__ __forceinline__ uint32_t top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) t = max(t, Vec<T>::top(raw[i]));
    return t;
  }
};
template <typename T>
__device__ __forceinline__ uint4 codes16(Sixteen<T> x, RowUnit u) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < Sixteen<T>::kVecs; ++i) {
    float v[Vec<T>::N];
    Vec<T>::unpack(x.raw[i], v);
    if (u.lift != 1.0f)
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) v[j] *= u.lift;
    uint32_t b[Vec<T>::N / 4];
    Vec<T>::codes(u, v, b);
#pragma unroll
    for (int j = 0; j < Vec<T>::N / 4; ++j) c[i * (Vec<T>::N / 4) + j] = b[j];
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

__device__ __forceinline__ void put_out(void* y, int dtype, int64_t at, float v) {
  if (dtype == TQ_DTYPE_F32) static_cast<float*>(y)[at] = v;
  else if (dtype == TQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(y)[at] = __float2half_rn(v);
}

// A CTA's tiles, in order: segment and row tile within it.
struct Tiles {
  int32_t left, seg, row_tile, row_tiles;
  __device__ __forceinline__ bool last_of_segment() const { return left == 1 || row_tile + 1 == row_tiles; }
  __device__ __forceinline__ void next() {
    --left;
    if (++row_tile == row_tiles) {
      row_tile = 0;
      ++seg;
    }
  }
};
// A place in the ring of weight stages.
struct Place {
  int32_t stages, at;
  uint32_t phase;
  __device__ __forceinline__ void skip(int32_t n) {
    at += n;
    while (at >= stages) {
      at -= stages;
      phase ^= 1u;
    }
  }
};

template <typename T, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 1)
    int8_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ Int8StreamArgs a,
                       int32_t stages) {
  __shared__ Shared sh;
  extern __shared__ uint8_t dyn_smem[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* btiles = ring + stages * kStageBytes;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  if (warp == 0) {
    // (a lane per barrier)
    if (lane < stages) {
      mbar_init(&sh.full[lane], 1);
      mbar_init(&sh.empty[lane], 1);
    } else if (lane >= 16 && lane < 18) {
      mbar_init(&sh.dfull[lane - 16], kIssuers);
      mbar_init(&sh.dempty[lane - 16], kEpilogue);
    } else if (lane == 18) {
      mbar_init(&sh.bfull, kQuantThreads);
      mbar_init(&sh.bempty, kIssuers + kEpilogue);   // (the epilogue reads the scales)
      sh.abort_flag = sh.quit = 0;
      for (int i = 0; i < kIssuers; ++i) mbar_init(&sh.drained[i], 1);
      if (CLUSTER) {
        const int tpr = threads_per_row(a.m);   // a word per row and warp of it from every CTA
        mbar_init(&sh.maxima, 1);
        mbar_init(&sh.sums, 1);
        mbar_arrive_expect_tx(&sh.maxima, 4 * a.parts * a.m * (tpr > 32 ? tpr / 32 : 1));
        mbar_arrive_expect_tx(&sh.sums, kRows * 16 * ((a.m + 3) / 4));
      }
    }
    fence_mbar_init();
  }
  if (warp == 1 && lane < kTok) sh.top[lane] = 0;
  __syncthreads();
  if (CLUSTER) cluster_arrive();   // every CTA's barriers are there
  // What a role reads before its wait for the kernel before is this call's
  // input.  Tensor memory is taken after the wait, and the next kernel let in
  // after that: of two that wait for one another, neither may hold columns
  // that the other still has to take.
  const bool routed = !CLUSTER && a.ids != nullptr, ahead = routed && a.mode == INT8_DOWN;
  if (!ahead) pdl_wait();
  if (routed) route(sh, a);
  if (ahead && warp != 0) pdl_wait();
  if (warp >= 1 && warp < 8) {
    if (warp == 2) {
      tmem_alloc(&sh.tmem_base, 2 * kAcc);
      tmem_relinquish();
      tc_fence_before();
    }
    named_bar_sync(3, 7 * 32);
    tc_fence_after();
    if (threadIdx.x == 64) pdl_launch_dependents();
  }
  volatile int* abortp = &sh.abort_flag;
  Tiles w;
  int k0 = 0, k1 = a.ksteps;
  w.row_tiles = a.row_tiles;
  if (CLUSTER) {
    w.left = 1;
    w.seg = 0;
    w.row_tile = blockIdx.x / a.parts;
    k0 = a.ksteps * rank / a.parts;
    k1 = a.ksteps * (rank + 1) / a.parts;
  } else {
    const int32_t segs = routed ? sh.nseg : a.segs ? __ldcg(a.nseg) : 1;
    const int32_t tiles = segs * a.row_tiles;
    const int32_t per = tiles / static_cast<int>(gridDim.x), rest = tiles - per * static_cast<int>(gridDim.x);
    const int32_t c = blockIdx.x, first = c * per + min(c, rest);
    w.left = per + (c < rest ? 1 : 0);
    w.seg = first / a.row_tiles;
    w.row_tile = first - w.seg * a.row_tiles;
  }
  const int32_t seg0 = w.seg;
  const int steps = k1 - k0;
  auto segment = [&](int32_t s) {
    return routed ? sh.segs[s] : a.segs ? __ldcg(a.segs + s) : make_int4(0, 0, a.m, 0);
  };
  auto slot_of = [&](int32_t row) { return routed ? sh.pairs[row] : __ldcg(a.pairs + row); };
  Place pos{stages, 0, 0};

  if (warp == 0) {
    if (lane == 0) {
      int filled = 0;   // copies sent
      bool ok = true;
#pragma unroll 1
      for (; ok && w.left > 0; w.next()) {
        const int expert = segment(w.seg).x;
#pragma unroll 1
        for (int kk = k0; kk < k1; ++kk) {
          if (filled >= stages && !mbar_wait(&sh.empty[pos.at], pos.phase ^ 1u, abortp)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.full[pos.at], kStageBytes);
          tma_load_3d(ring + pos.at * kStageBytes, &tm_w, &sh.full[pos.at], kk * kStep, w.row_tile * kRows, expert);
          pos.skip(1);
          ++filled;
        }
      }
      sh.filled = filled;
    }
    __syncwarp();
  } else if (warp <= kIssuers) {
    // The whole warp walks, one elected lane issues: values that are the same
    // in every lane stay in the uniform registers that the MMA takes them from.
    const int me = warp - 1;
    int ti = 0, turn3 = 0;   // whose turn the tile's first k step is
    bool ok = true, fresh = true;   // the first tile of a segment
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abortp)) != 0;
    };
#pragma unroll 1
    for (; ok && w.left > 0; w.next(), ++ti) {
      const int turn = w.seg - seg0, db = ti & 1;
      if (fresh && !wait(&sh.bfull, turn & 1)) break;
      fresh = false;
      if (!wait(&sh.dempty[db], ((ti >> 1) & 1) ^ 1u)) break;
      tc_fence_after();
      const uint32_t d_addr = sh.tmem_base + db * kAcc + me * kTok;
      const int first = me >= turn3 ? me - turn3 : me - turn3 + kIssuers;   // its first k step of this tile
      Place p = pos;
      p.skip(first);
#pragma unroll 1
      for (int kk = first; kk < steps; kk += kIssuers) {
        ok = wait(&sh.full[p.at], p.phase);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = sdesc_k128(smem_u32(ring + p.at * kStageBytes));
        const uint64_t bd = sdesc_k128(smem_u32(btiles + kk * kTileB));
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < kStep / 32; ++q)   // (32 bytes on: 2 units of 16)
            mma_i8(d_addr, ad + q * 2, bd + q * 2, idesc_i8(kRows, kTok), (kk > first || q) ? 1u : 0u);
          mma_commit(&sh.empty[p.at]);
        }
        __syncwarp();
        p.skip(kIssuers);
      }
      if (!ok) break;
      pos.skip(steps);
      turn3 = (turn3 + steps) % kIssuers;
      fresh = w.last_of_segment();
      if (elect_one()) {
        mma_commit(&sh.dfull[db]);
        if (fresh) mma_commit(&sh.bempty);
      }
      __syncwarp();
    }
    // MMAs and the arrivals of the commits above end before the CTA does: a
    // late arrival would meet the barriers of the CTA that comes after it
    if (elect_one()) {
      mma_commit(&sh.drained[me]);
      int8_drain_wait(&sh.drained[me], 0);
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- the tokens' codes
    const int q = threadIdx.x - 256;
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * static_cast<int>(sizeof(T)) % 16 == 0;
    // Where a wait ran out they stop together, before they report the segment:
    // the barrier counts one report a thread and phase, and waits for what it
    // guards alone keep a report out of the phase before.
    bool ok = true, go = true;
#pragma unroll 1
    for (int32_t s = seg0, n = (w.row_tile + w.left + a.row_tiles - 1) / a.row_tiles; go && n > 0 && w.left > 0;
         ++s, --n) {
      const int turn = s - seg0;
      const int4 sg = segment(s);
      const int tpr = threads_per_row(sg.z);
      const int r = q / tpr, i0 = q - r * tpr;
      const bool live = r < sg.z;
      const int row = sg.y + r;
      const int64_t from = !live ? 0 : a.mode == INT8_UP ? slot_of(row) / a.topk : row;
      const T* x = static_cast<const T*>(a.x) + from * a.ldx;
      const int c0 = k0 * (kStep / 16), c1 = live ? min(k1 * (kStep / 16), a.k / 16) : 0;   // chunks of 16
      Sixteen<T> hold[kHold];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < kHold; ++j) {
        const int c = c0 + i0 + j * tpr;
        if (c < c1) hold[j].load(x + static_cast<int64_t>(c) * 16, wide);
      }
      if (ok) ok = mbar_wait(&sh.bempty, (turn & 1) ^ 1u, abortp);
#pragma unroll
      for (int j = 0; j < kHold; ++j)
        if (c0 + i0 + j * tpr < c1) top = max(top, hold[j].top());
#pragma unroll 1
      for (int c = c0 + i0 + kHold * tpr; c < c1; c += 2 * tpr) {
        Sixteen<T> v, u;
        v.load(x + static_cast<int64_t>(c) * 16, wide);
        const int d = c + tpr < c1 ? c + tpr : c;
        u.load(x + static_cast<int64_t>(d) * 16, wide);
        top = max(top, max(v.top(), u.top()));
      }
      // the row's largest: within the warp, then among warps and CTAs
      const int width = min(tpr, 32);
      for (int o = width >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const bool leader = live && (lane & (width - 1)) == 0;
      uint32_t row_top = 0;
      if (CLUSTER) {
        cluster_wait();
        const int at = tpr > 32 ? q >> 5 : r;
        if (leader)
          for (int p = 0; p < a.parts; ++p)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(
                             in_cta(&sh.tops[rank][at], p)),
                         "r"(top), "r"(in_cta(&sh.maxima, p))
                         : "memory");
        mbar_wait_cluster(&sh.maxima, 0, abortp);   // (where it runs out the epilogue stores nothing)
        if (live) {
          const int n_at = tpr > 32 ? tpr / 32 : 1, at0 = tpr > 32 ? r * n_at : r;
          for (int p = 0; p < a.parts; ++p)
            for (int i = 0; i < n_at; ++i)
              row_top = max(row_top, *reinterpret_cast<volatile uint32_t*>(&sh.tops[p][at0 + i]));
        }
      } else {
        if (leader) atomicMax(&sh.top[r], top);
        if (!ok) sh.quit = 1;
        named_bar_sync(2, kQuantThreads);
        go = *const_cast<volatile int*>(&sh.quit) == 0;   // (the same for all: written before the barrier only)
        if (live) row_top = *reinterpret_cast<volatile uint32_t*>(&sh.top[r]);
      }
      const RowUnit u(Vec<T>::top_f32(row_top));
      if (i0 == 0 && live) {
        if (!u.finite) raise_status(TQ_DEV_NONFINITE);
        sh.sx[r] = u.scale;
        if (a.mode == INT8_DOWN) {
          sh.slot[r] = slot_of(row);
          sh.tw[r] = routed ? sh.row_w[row] : __ldcg(a.row_w + row);
        }
      }
      // (rows and columns without a value keep what was there: it meets
      // outputs that are not stored, and weights that the copy filled with 0)
      uint8_t* b = btiles + (r & 15) * kStep;
      auto put = [&](int c, const Sixteen<T>& v) {
        const int at = c - c0;   // k step and 16-byte piece of the tile, swizzled
        *reinterpret_cast<uint4*>(b + (at >> 3) * kTileB + (((at & 7) ^ (r & 7)) << 4)) = codes16<T>(v, u);
      };
#pragma unroll
      for (int j = 0; j < kHold; ++j)
        if (c0 + i0 + j * tpr < c1) put(c0 + i0 + j * tpr, hold[j]);
#pragma unroll 1
      for (int c = c0 + i0 + kHold * tpr; c < c1; c += tpr) {
        Sixteen<T> v;
        v.load(x + static_cast<int64_t>(c) * 16, wide);
        put(c, v);
      }
      fence_proxy_async_smem();
      if (!CLUSTER) {
        named_bar_sync(2, kQuantThreads);   // every thread has read its row's maximum
        if (q < kTok) sh.top[q] = 0;
      }
      if (go && !(a.test_withhold && warp == 8 && turn == 0 && rank == 0)) mbar_arrive(&sh.bfull);
      if (CLUSTER) cluster_arrive_relaxed();
    }
  } else {
    // ---- epilogue
    const int t = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int accs = steps < kIssuers ? steps : kIssuers;
    int ti = 0, turn3 = 0;
    bool ok = true, fresh = true;
    int4 sg = make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (; w.left > 0; w.next(), ++ti) {
      const int turn = w.seg - seg0, db = ti & 1;
      if (fresh) {
        sg = segment(w.seg);
        ok = ok && mbar_wait(&sh.bfull, turn & 1, abortp);   // the scales
        fresh = false;
      }
      const int row = w.row_tile * kRows + t;
      const float sw = row < a.n ? __ldcg(a.wscale + static_cast<int64_t>(sg.x) * a.n + row) : 0.0f;
      ok = ok && mbar_wait(&sh.dfull[db], (ti >> 1) & 1, abortp);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok && !CLUSTER) break;
      tc_fence_after();
      int32_t acc[kTok];
#pragma unroll
      for (int j = 0; j < kTok; ++j) acc[j] = 0;
      if (ok)
#pragma unroll 1
        for (int i = 0; i < accs; ++i) {
          uint32_t d[kTok];
          tmem_ld16(sh.tmem_base + lane_base + db * kAcc + (turn3 + i) % kIssuers * kTok, d);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < kTok; ++j) acc[j] += static_cast<int32_t>(d[j]);
        }
      turn3 = (turn3 + steps) % kIssuers;
      if (CLUSTER) {
        // rows belong to the CTAs in turn, 128 / parts each; what is sent is
        // counted by its owner, so it is sent after a timeout too
        cluster_wait();
        const int per = kRows / a.parts, owner = t / per;
        const uint32_t to = in_cta(&sh.part[(rank * per + (t - owner * per)) * kPartRow], owner);
        const uint32_t bar = in_cta(&sh.sums, owner);
#pragma unroll
        for (int j = 0; j < kTok; j += 4)
          if (j < sg.z)
            asm volatile(
                "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                    to + j * 4),
                "r"(acc[j]), "r"(acc[j + 1]), "r"(acc[j + 2]), "r"(acc[j + 3]), "r"(bar)
                : "memory");
        cluster_arrive_relaxed();   // (these are the last)
        int never = 0;   // (no giving up for an abort: others' stores may be on their way here)
        const bool got = mbar_wait_cluster(&sh.sums, 0, &never);
        if (!got) *abortp = 1;
        const int row_base = w.row_tile * kRows + rank * per;
        for (int i = ok && got && !*abortp ? t : INT32_MAX; i < per * (kTok / 4); i += kEpilogue) {
          const int rl = i % per, j0 = i / per * 4, out_row = row_base + rl;
          if (out_row >= a.n || j0 >= sg.z) continue;
          int4 sum = make_int4(0, 0, 0, 0);
          for (int p = 0; p < a.parts; ++p) {
            const int4 v = *reinterpret_cast<const int4*>(&sh.part[(p * per + rl) * kPartRow + j0]);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
          }
          const float osw = __ldcg(a.wscale + out_row);
          const int32_t v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j0 + j < sg.z)
              put_out(a.y, a.dtype, static_cast<int64_t>(j0 + j) * a.n + out_row,
                      __fmul_rn(__fmul_rn(static_cast<float>(v[j]), sh.sx[j0 + j]), osw));
        }
      } else {
        tc_fence_before();
        mbar_arrive(&sh.dempty[db]);
        if (row < a.n) {
#pragma unroll
          for (int j = 0; j < kTok; ++j) {
            if (j >= sg.z) break;
            const float f = __fmul_rn(__fmul_rn(static_cast<float>(acc[j]), sh.sx[j]), sw);
            if (a.mode == INT8_DOWN) {
              static_cast<float*>(a.y)[static_cast<int64_t>(sh.slot[j]) * a.n + row] = __fmul_rn(f, sh.tw[j]);
            } else {
              const float g = f < 0.0f ? 0.0f : f;   // (a NaN stays)
              put_out(a.y, a.mode == INT8_UP ? TQ_DTYPE_BF16 : a.dtype, static_cast<int64_t>(sg.y + j) * a.n + row,
                      a.mode == INT8_UP ? __fmul_rn(g, g) : f);
            }
          }
        }
        if (w.last_of_segment()) {
          mbar_arrive(&sh.bempty);
          fresh = true;
        }
      }
    }
  }

  if (CLUSTER) {
    // No CTA leaves before every other has sent what it sends: one whose wait
    // ran out would be written to after its end.
    if (warp < 4) {
      cluster_wait();
      cluster_arrive_relaxed();
    }
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(sh.tmem_base, 2 * kAcc);
  // Where a wait ran out, copies may be in flight, and what other CTAs sent.
  // (Not before here: a role may give up after the last copy was sent.)
  if (threadIdx.x == 0 && *abortp) {
    int8_land_copies(sh.full, stages, sh.filled);
    if (CLUSTER) {
      int8_drain_wait(&sh.maxima, 0);
      int8_drain_wait(&sh.sums, 0);
    }
  }
}

template <typename T>
cudaError_t launch_as(const CUtensorMap& tw, const Int8StreamArgs& a, int64_t most_tiles, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = once_per_device(attr_done, [] {
    cudaError_t r = cudaFuncSetAttribute(int8_stream_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSpace + 1024);
    if (r != cudaSuccess) return r;
    return cudaFuncSetAttribute(int8_stream_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSpace + 1024);
  });
  if (e != cudaSuccess) return e;
  const int part_steps = (a.ksteps + a.parts - 1) / a.parts, b_bytes = part_steps * kTileB;
  int stages = (kSpace - b_bytes) / kStageBytes;
  if (stages > kMaxStages) stages = kMaxStages;
  if (a.parts > 1 && stages >= part_steps) stages = part_steps;   // (none is used again)
  else stages -= stages % kIssuers;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(b_bytes) + static_cast<size_t>(stages) * kStageBytes + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  // set up while the kernel before still runs; the kernel waits for its end
  // before its first load of tokens, segments or weight
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n++].val.programmaticStreamSerializationAllowed = 1;
  if (a.parts > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(a.parts);
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (a.parts > 1) {
    cfg.gridDim = dim3(static_cast<unsigned>(a.row_tiles * a.parts));
    e = cudaLaunchKernelEx(&cfg, int8_stream_kernel<T, true>, tw, a, stages);
  } else {
    cfg.gridDim = dim3(static_cast<unsigned>(most_tiles < sms ? most_tiles : sms));
    e = cudaLaunchKernelEx(&cfg, int8_stream_kernel<T, false>, tw, a, stages);
  }
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace

bool int8_stream_fits(int64_t k) { return (k + kStep - 1) / kStep * kTileB <= kSpace - 4 * kStageBytes; }

int int8_stream_parts(int64_t row_tiles, int64_t ksteps, int sms) {
  int parts = 1;
  while (parts < kMaxParts && row_tiles * parts * 2 <= sms && ksteps >= parts * 4) parts *= 2;
  return parts;
}

cudaError_t launch_int8_stream(int xdtype, const CUtensorMap& tw, const Int8StreamArgs& a, int64_t most_tiles, int sms,
                               cudaStream_t st) {
  switch (xdtype) {
    case TQ_DTYPE_F32: return launch_as<float>(tw, a, most_tiles, sms, st);
    case TQ_DTYPE_BF16: return launch_as<__nv_bfloat16>(tw, a, most_tiles, sms, st);
    default: return launch_as<__half>(tw, a, most_tiles, sms, st);
  }
}

}  // namespace tq4
