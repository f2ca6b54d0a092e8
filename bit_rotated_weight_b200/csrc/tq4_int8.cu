// The int8 format (int8 codes, one fp32 scale per row): its quantizer and the
// way back, the linear layer and the MoE on it.
//
// A row x quantizes to q_i = round(127 x_i / max|x|), ties to even, with scale
// = fp32(max|x| / 127); the row it stands for is scale * q.  The rounding is
// that of the real quotient, not of some fp32 product: half of a row's largest
// value lies exactly on a border (63.5), so a quotient that is off by one unit
// would round by chance there.
#include <type_traits>

#include "tq4_int8_rows.cuh"

#define TQ_API extern "C" __attribute__((visibility("default")))

namespace tq4 {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}

struct RowsArgs {
  const void* x;
  int64_t ldx, k, rows;
  int8_t* q;                 // [rows][k], or sorted rows (scatter)
  float* scale;
  const int32_t* rows_dev;   // rows past *rows_dev are left alone (nullptr: none)
  // scatter: row t goes to the sorted rows of its topk slots, whose slot
  // numbers and weights are left in pairs and row_w; each expert's next row is
  // cursor[expert].  (The order of an expert's rows may differ from run to
  // run; a row's results do not depend on its place.)
  const int32_t* ids;
  int32_t topk, num_experts;
  int32_t* cursor;
  int32_t* pairs;
  const float* topk_w;
  float* row_w;
};

// Counts each expert's slots and writes the segments (at most `chunk` rows of
// one expert), their number, the number of rows, and each expert's first row
// (the scatter's cursors).  By one block; `count`: an int per expert, holds the
// first rows in the end.
struct SegmentArgs {
  const int32_t* ids;
  int64_t slots;
  int32_t num_experts, chunk;
  int32_t* cursor;
  int4* segs;
  int32_t* nseg;
  int32_t* nrows;
};
template <int THREADS>
__device__ __forceinline__ void segments_of(const SegmentArgs& a, int32_t* count) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int32_t s_rows[kWarps], s_segs[kWarps];
  __shared__ int32_t s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < a.num_experts; e += THREADS) count[e] = 0;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int64_t p0 = tid; p0 < a.slots; p0 += 8 * THREADS) {   // (eight loads in flight a thread)
    int32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = p0 + j * THREADS < a.slots ? __ldcg(a.ids + p0 + j * THREADS) : INT32_MIN;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (e[j] >= 0 && e[j] < a.num_experts) atomicAdd(&count[e[j]], 1);
      else if (p0 + j * THREADS < a.slots) s_bad = 1;
    }
  }
  __syncthreads();
  int32_t rows0 = 0, segs0 = 0;   // of the experts before this pass
  for (int e0 = 0; e0 < a.num_experts; e0 += THREADS) {
    const int e = e0 + tid;
    const int32_t c = e < a.num_experts ? count[e] : 0;
    const int32_t ns = (c + a.chunk - 1) / a.chunk;
    int32_t rows = c, nsegs = ns;   // inclusive scans: warp, then block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t r = __shfl_up_sync(0xFFFFFFFFu, rows, o), s = __shfl_up_sync(0xFFFFFFFFu, nsegs, o);
      if (lane >= o) {
        rows += r;
        nsegs += s;
      }
    }
    if (lane == 31) {
      s_rows[warp] = rows;
      s_segs[warp] = nsegs;
    }
    __syncthreads();
    int32_t total_r = 0, total_s = 0, before_r = rows0, before_s = segs0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        before_r += s_rows[w];
        before_s += s_segs[w];
      }
      total_r += s_rows[w];
      total_s += s_segs[w];
    }
    const int32_t row = before_r + rows - c, seg = before_s + nsegs - ns;
    if (e < a.num_experts) {
      a.cursor[e] = row;
      count[e] = row;
      for (int32_t i = 0; i < ns; ++i)
        a.segs[seg + i] = make_int4(e, row + i * a.chunk, min(a.chunk, c - i * a.chunk), 0);
    }
    rows0 += total_r;
    segs0 += total_s;
    __syncthreads();
  }
  if (tid == 0) {
    *a.nseg = segs0;
    *a.nrows = rows0;
    if (s_bad) raise_status(TQ_DEV_BAD_ROUTING);
  }
}

// With `pairs` the rows are given out here: the slot and weight of each sorted
// row.
__global__ void __launch_bounds__(1024) int8_segments_kernel(const __grid_constant__ SegmentArgs a, const float* topk_w,
                                                             int32_t* pairs, float* row_w) {
  extern __shared__ int32_t count[];
  pdl_launch_dependents();
  pdl_wait();
  segments_of<1024>(a, count);
  if (pairs)
    for (int64_t p = threadIdx.x; p < a.slots; p += 1024) {
      const int32_t e = a.ids[p];
      if (e < 0 || e >= a.num_experts) continue;
      const int32_t at = atomicAdd(&count[e], 1);
      pairs[at] = static_cast<int32_t>(p);
      row_w[at] = topk_w[p];
    }
}

constexpr int kRowThreads = 256;

// The destination rows of a scattered row (one expert slot each).
// `threads` threads work on the row; topk (up to 64) may be more.
__device__ __forceinline__ void take_rows(const RowsArgs& a, int64_t row, int lane, int threads, int32_t* s_at) {
  for (int j = lane; j < a.topk; j += threads) {
    const int64_t slot = row * a.topk + j;
    const int32_t e = a.ids[slot];
    int32_t at = -1;
    if (e >= 0 && e < a.num_experts) {
      at = atomicAdd(a.cursor + e, 1);
      a.pairs[at] = static_cast<int32_t>(slot);
      a.row_w[at] = a.topk_w[slot];
    }
    s_at[j] = at;
  }
}
__device__ __forceinline__ void put_scale(const RowsArgs& a, int64_t row, int lane, int threads, const int32_t* s_at,
                                          float scale) {
  if (a.ids) {
    for (int j = lane; j < a.topk; j += threads)
      if (s_at[j] >= 0) a.scale[s_at[j]] = scale;
  } else if (lane == 0) {
    a.scale[row] = scale;
  }
}

// How a row finds its places: it has one (its own), one per slot, taken from the
// experts' cursors, or counts them itself among at most kCountSlots ids (a
// kernel less, as the grid's last block writes the segments meanwhile: 134
// tokens x 4 of 8 small experts 20.2 -> 16.5 us, at 1996 slots 26.5 -> 24.7).
enum Places { kOwnRow = 0, kCursors = 1, kCounts = 2 };
constexpr int kCountSlots = 2048;

// The places of the block's rows: the slots with a smaller id, and those with
// the same one earlier.  A warp a slot.
__device__ __forceinline__ void count_rows(const RowsArgs& a, int64_t row0, int rows, int32_t* ids,
                                           int32_t (*s_at)[64]) {
  const int slots = static_cast<int>(a.rows) * a.topk, lane = threadIdx.x & 31;
  for (int p = threadIdx.x; p < slots; p += kRowThreads) ids[p] = __ldcg(a.ids + p);
  __syncthreads();
  for (int q = threadIdx.x >> 5; q < rows * a.topk; q += kRowThreads / 32) {
    const int sub = q / a.topk, j = q - sub * a.topk;
    const int slot = static_cast<int>(row0 + sub) * a.topk + j;
    if (row0 + sub >= a.rows) break;
    const int32_t e = ids[slot];
    const bool valid = e >= 0 && e < a.num_experts;
    int at = 0;
#pragma unroll 4
    for (int p = lane; p < slots; p += 32) at += (ids[p] >= 0 && ids[p] < e) || (ids[p] == e && p < slot) ? 1 : 0;
    at = __reduce_add_sync(0xFFFFFFFFu, at);
    if (lane == 0) {
      s_at[sub][j] = valid ? at : -1;
      if (valid) {
        a.pairs[at] = slot;
        a.row_w[at] = a.topk_w[slot];
      }
    }
  }
  __syncthreads();
}

// TPR threads hold a row of at most TPR * NV 16-byte vectors in registers: one
// pass over the data, all of a thread's loads in flight at once.  14336 x 4096
// fp32 in 43 us: 294 MB, 6.9 TB/s (235 MB of them from DRAM, at 68 % of its
// nominal rate; the codes stay in L2).  bf16 in 33 us: 176 MB, 5.4 TB/s, but only
// 126 MB from and to DRAM, 45 % of its rate; there the issue slots (71 % of the
// active cycles) and the integer pipe (61 %) come before it, at 36 warps an SM.
template <typename T, int TPR, int NV, int PLACES>
__global__ void __launch_bounds__(kRowThreads)
    int8_rows_kernel(const __grid_constant__ RowsArgs a, const __grid_constant__ SegmentArgs sa) {
  using V = Vec<T>;
  constexpr bool SCATTER = PLACES != kOwnRow;
  extern __shared__ int32_t s_ids[];
  constexpr int kRowsPerBlock = kRowThreads / TPR;
  __shared__ uint32_t s_top[kRowThreads / 32];
  __shared__ int32_t s_at[SCATTER ? kRowsPerBlock : 1][64];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  if (PLACES == kCounts && blockIdx.x == gridDim.x - 1) {
    segments_of<kRowThreads>(sa, s_ids);
    return;
  }
  const int64_t rows = a.rows_dev ? __ldcg(a.rows_dev) : a.rows;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + sub;
  const bool live = row < rows;
  if (TPR == 32 ? !live : static_cast<int64_t>(blockIdx.x) * kRowsPerBlock >= rows) return;
  const int nvec = static_cast<int>(a.k) / V::N;
  const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + (live ? row : 0) * a.ldx);
  uint4 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    raw[i] = live && lane + i * TPR < nvec ? __ldcs(x + lane + i * TPR) : make_uint4(0, 0, 0, 0);
  if (PLACES == kCursors && live) take_rows(a, row, lane, TPR, s_at[sub]);
  if (PLACES == kCounts) count_rows(a, static_cast<int64_t>(blockIdx.x) * kRowsPerBlock, kRowsPerBlock, s_ids, s_at);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) top = max(top, V::top(raw[i]));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) top = max(top, s_top[sub * (TPR / 32) + w]);
  } else {
    __syncwarp();
  }
  if (!live) return;
  const RowUnit u(V::top_f32(top));
  if (!u.finite && lane == 0) raise_status(TQ_DEV_NONFINITE);
  put_scale(a, row, lane, TPR, s_at[SCATTER ? sub : 0], u.scale);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = lane + i * TPR;
    if (at >= nvec) break;
    float v[V::N];
    V::unpack(raw[i], v);
    if (u.lift != 1.0f)
#pragma unroll
      for (int j = 0; j < V::N; ++j) v[j] *= u.lift;
    uint32_t c[V::N / 4];
    V::codes(u, v, c);
    auto put = [&](int64_t to) {
      uint32_t* q = reinterpret_cast<uint32_t*>(a.q + to * a.k) + static_cast<int64_t>(at) * (V::N / 4);
      if constexpr (V::N == 8) *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[1]);
      else *q = c[0];
    };
    if constexpr (SCATTER) {
      for (int j = 0; j < a.topk; ++j)
        if (s_at[sub][j] >= 0) put(s_at[sub][j]);
    } else {
      put(row);
    }
  }
}

// Rows of any length and alignment, read twice.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) int8_rows_any_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ uint32_t s_top[kRowThreads / 32];
  __shared__ int32_t s_at[64];
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  if (a.rows_dev && row >= __ldcg(a.rows_dev)) return;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  uint32_t top = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.k; i += kRowThreads) top = max(top, __float_as_uint(fabsf(to_f32(x[i]))));
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  if (a.ids) take_rows(a, row, threadIdx.x, kRowThreads, s_at);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) top = max(top, s_top[w]);
  const RowUnit u(top);
  if (!u.finite && threadIdx.x == 0) raise_status(TQ_DEV_NONFINITE);
  put_scale(a, row, threadIdx.x, kRowThreads, s_at, u.scale);
#pragma unroll 2
  for (int64_t i = 4 * threadIdx.x; i < a.k; i += 4 * kRowThreads) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = to_f32(x[i + j]) * u.lift;
    uint32_t c[1];
    if constexpr (sizeof(T) == 2) codes_of_16(u, v, c);
    else codes_of_32(u, v, c);
    if (a.ids) {
      for (int j = 0; j < a.topk; ++j)
        if (s_at[j] >= 0) *reinterpret_cast<uint32_t*>(a.q + s_at[j] * a.k + i) = c[0];
    } else {
      *reinterpret_cast<uint32_t*>(a.q + row * a.k + i) = c[0];
    }
  }
}

constexpr int kDeqGroups = 4;   // groups of 4 codes per thread

// Back to fp32.  Bound by DRAM: 14336 x 4096 in 46 us, 6.4 TB/s (the codes
// come from L2 in part).
__global__ void __launch_bounds__(256) int8_dequantize_kernel(const int8_t* q, const float* scale, float* out,
                                                              int64_t rows, int32_t kg) {
  // kg: groups of 4 codes in a row.  The block's first group is located with
  // one 64-bit division, the others from there.
  pdl_wait();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kDeqGroups);
  const int64_t row0 = first / kg, total = rows * kg;
  const uint32_t col0 = static_cast<uint32_t>(first - row0 * kg);
  char4 c[kDeqGroups];
  float s[kDeqGroups];
#pragma unroll
  for (int j = 0; j < kDeqGroups; ++j) {
    const uint32_t at = threadIdx.x + 256 * j;
    if (first + at >= total) break;
    c[j] = __ldcs(reinterpret_cast<const char4*>(q) + first + at);
    s[j] = scale[row0 + (col0 + at) / static_cast<uint32_t>(kg)];
  }
#pragma unroll
  for (int j = 0; j < kDeqGroups; ++j) {
    const uint32_t at = threadIdx.x + 256 * j;
    if (first + at >= total) break;
    __stcs(reinterpret_cast<float4*>(out) + first + at,
           make_float4(__fmul_rn(static_cast<float>(c[j].x), s[j]), __fmul_rn(static_cast<float>(c[j].y), s[j]),
                       __fmul_rn(static_cast<float>(c[j].z), s[j]), __fmul_rn(static_cast<float>(c[j].w), s[j])));
  }
}

// y[t] = T(sum over the slots of token t, in order, of their weighted row z).
// Four outputs a thread; the rows of up to eight slots are requested before
// the first is added.  Bound by DRAM: 4096 tokens x 6 slots of 2688 in 43 us,
// 6.6 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) int8_combine_kernel(const float* z, const int32_t* ids, int64_t m, int32_t topk,
                                                           int32_t hg, int32_t num_experts, T* y) {
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= m * hg) return;
  const int64_t t = i / hg;
  const int32_t n = static_cast<int32_t>(i - t * hg);
  const float4* zt = reinterpret_cast<const float4*>(z) + t * topk * hg + n;
  const int32_t* idt = ids + t * topk;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = 0; j0 < topk; j0 += 8) {
    float4 v[8];
    int32_t e[8];
    // (a skipped slot's row is read too, whatever it holds: a load that waits
    // for its id would come a memory latency later)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      e[j] = -1;
      if (j0 + j < topk) {
        v[j] = __ldcs(zt + static_cast<int64_t>(j0 + j) * hg);
        e[j] = idt[j0 + j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e[j] >= 0 && e[j] < num_experts) {
        s.x = __fadd_rn(s.x, v[j].x);
        s.y = __fadd_rn(s.y, v[j].y);
        s.z = __fadd_rn(s.z, v[j].z);
        s.w = __fadd_rn(s.w, v[j].w);
      }
  }
  uint2 o;
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 lo = __floats2half2_rn(s.x, s.y), hi = __floats2half2_rn(s.z, s.w);
    o = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    o = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
  *(reinterpret_cast<uint2*>(y) + i) = o;
}

template <typename T, int TPR, int NV>
cudaError_t launch_rows_as(const RowsArgs& a, cudaLaunchConfig_t& cfg, const SegmentArgs* sa = nullptr) {
  cfg.gridDim = dim3(static_cast<unsigned>((a.rows + kRowThreads / TPR - 1) / (kRowThreads / TPR)));
  const SegmentArgs none{};
  if constexpr (TPR >= 128)
    if (sa) {
      cfg.gridDim.x += 1;
      cfg.dynamicSmemBytes = 4 * static_cast<size_t>(sa->slots > sa->num_experts ? sa->slots : sa->num_experts);
      return cudaLaunchKernelEx(&cfg, int8_rows_kernel<T, TPR, NV, kCounts>, a, *sa);
    }
  return a.ids ? cudaLaunchKernelEx(&cfg, int8_rows_kernel<T, TPR, NV, kCursors>, a, none)
               : cudaLaunchKernelEx(&cfg, int8_rows_kernel<T, TPR, NV, kOwnRow>, a, none);
}

// Whether the rows can count their places themselves (those that do are long
// or few enough for 128 threads each).
template <typename T>
bool rows_count(const RowsArgs& a) {
  return a.rows * a.topk <= kCountSlots && a.k / Vec<T>::N <= 256 * 8 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
         a.ldx % Vec<T>::N == 0;
}

template <typename T>
cudaError_t launch_rows_of(const RowsArgs& a, cudaLaunchConfig_t& cfg, const SegmentArgs* sa) {
  const int64_t nvec = a.k / Vec<T>::N;
  const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % Vec<T>::N == 0;
  // Many rows: a warp each up to 4 KB (24576 x 1856 bf16 24.0 us, 28.8 with two
  // warps), four warps up to 16 KB (14336 x 4096 bf16 33.6 us, 78.7 with one;
  // fp32 45.6 us, 48.6 with eight).  Few: as many threads as there are pieces.
  if (wide && !sa && a.rows >= 148 * 8) {
    if (nvec <= 32 * 4) return launch_rows_as<T, 32, 4>(a, cfg);
    if (nvec <= 32 * 8) return launch_rows_as<T, 32, 8>(a, cfg);
    if (nvec <= 128 * 4) return launch_rows_as<T, 128, 4>(a, cfg);
    if (nvec <= 128 * 8) return launch_rows_as<T, 128, 8>(a, cfg);
  }
  if (wide && nvec <= 128) return launch_rows_as<T, 128, 1>(a, cfg, sa);
  if (wide && nvec <= 256 * 2) return launch_rows_as<T, 256, 2>(a, cfg, sa);
  if (wide && nvec <= 256 * 4) return launch_rows_as<T, 256, 4>(a, cfg, sa);
  if (wide && nvec <= 256 * 8) return launch_rows_as<T, 256, 8>(a, cfg, sa);
  cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
  return cudaLaunchKernelEx(&cfg, int8_rows_any_kernel<T>, a);
}

// A launch that may be set up while the kernel before it still runs (every
// kernel here waits for its end before its first load or store, and reads by
// plain loads: read-only ones are for what nothing writes while a kernel runs).
// A plain launch costs the host a microsecond more.
void launch_early(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, unsigned grid, unsigned threads, size_t smem,
                  cudaStream_t st) {
  cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
}

cudaError_t launch_rows(int dtype, const RowsArgs& a, cudaStream_t st, const SegmentArgs* sa = nullptr) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_early(cfg, attr, 1, kRowThreads, 0, st);   // (the grid is set below)
  const cudaError_t e = dtype == TQ_DTYPE_F32    ? launch_rows_of<float>(a, cfg, sa)
                        : dtype == TQ_DTYPE_BF16 ? launch_rows_of<__nv_bfloat16>(a, cfg, sa)
                                                 : launch_rows_of<__half>(a, cfg, sa);
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ host
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int rc_of(cudaError_t e) { return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA; }
bool aligned_elem(const void* p, int dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == TQ_DTYPE_F32 ? 4 : 2) == 0;
}
bool dtype_ok(int dtype) { return dtype == TQ_DTYPE_F32 || dtype == TQ_DTYPE_BF16 || dtype == TQ_DTYPE_F16; }

int weight_ok(const tq4_1s_int8_weight* w, bool need_ptrs) {
  if (!w || w->n <= 0 || w->k <= 0 || w->k % 32 != 0 || w->num_experts <= 0 || w->reserved != 0)
    return TQ_ERR_INVALID_ARG;
  if (w->n > (1ll << 30) || w->k > kInt8MaxK || w->num_experts > 4096) return TQ_ERR_INVALID_ARG;
  if (need_ptrs) {
    if (!w->q || !w->wscale) return TQ_ERR_INVALID_ARG;
    if (!aligned16(w->q) || !aligned16(w->wscale)) return TQ_ERR_ALIGNMENT;
  }
  return TQ_OK;
}

constexpr int64_t kMaxTiles = 1 << 30;

// How a dense product is run: tokens a tile, CTAs.
struct Plan {
  int nt, grid;
  int64_t row_tiles, tok_tiles, ksteps;
};
// The tile width with the least waves x time of a tile.  A tile's time goes
// about as 232 + NT (7 us at NT = 32, 8.2 at 128, 12.2 at 256, for k = 4096):
// small tiles are bound by the latency of a k step, and pay while they fit in
// one wave (512 x 4096 x 4096: 13.5 us at 128, 16.8 at 256, 19.7 at 64), large
// ones by the MMAs.
Plan plan_dense(int64_t m, int64_t n, int64_t k, int sms) {
  Plan p;
  int64_t best = INT64_MAX;
  for (const int nt : {16, 32, 64, 128, 256}) {
    if (nt == 16 ? m > 16 : nt > 32 && m <= nt / 2) continue;
    const int64_t tiles = (n + 127) / 128 * ((m + nt - 1) / nt), time = (tiles + sms - 1) / sms * (232 + nt);
    if (time < best) {
      best = time;
      p.nt = nt;
    }
  }
  p.row_tiles = (n + 127) / 128;
  p.tok_tiles = (m + p.nt - 1) / p.nt;
  p.ksteps = (k + 127) / 128;
  int64_t tiles = p.row_tiles * p.tok_tiles;
  p.grid = static_cast<int>(tiles < sms ? tiles : sms);
  // Many tiles: two CTAs share one of 256 rows x 256 tokens (8192 x 14336 x
  // 4096: 353 us sustained, 400 without; in one wave the launch costs more
  // than the copies saved: 1024 x 4096 x 4096 22.4 and 20.5).
  if (p.nt == 256 && (n + 255) / 256 * p.tok_tiles > sms / 2) {
    p.nt = kInt8Pair;
    p.row_tiles = (n + 255) / 256;
    tiles = p.row_tiles * p.tok_tiles;
    p.grid = 2 * static_cast<int>(tiles < sms / 2 ? tiles : sms / 2);
  }
  return p;
}

// Few tokens: one kernel that streams the weight and quantizes x itself.
bool streams(int64_t m, int64_t k) { return m <= kStreamTokens && int8_stream_fits(k); }

struct LinearLayout {
  size_t xq, xscale, total;
};
LinearLayout linear_layout(int64_t m, int64_t k) {
  LinearLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.xq = take(static_cast<size_t>(m) * static_cast<size_t>(k));
  L.xscale = take(static_cast<size_t>(m) * 4);
  L.total = off;
  return L;
}

struct MoeLayout {
  size_t cursor, segs, nseg, nrows, pairs, row_w, xq, xscale, h, hq, hscale, z, total;
  int nt;
  int64_t slots, maxseg;
};
MoeLayout moe_layout(int64_t m, int32_t topk, int64_t experts, int64_t H, int64_t I) {
  MoeLayout L{};
  L.slots = m * topk;
  // Rows of a segment, by the mean rows of an expert.  While the weight's
  // stream bounds the layer the width hardly matters (128 experts, 512 tokens
  // x 6: 237 us at 64 and 128, 243 at 32, 261 at 256); from 136 on it is the MMAs
  // (4096 tokens: 456 us at 256, 507 at 128; 2048: 351 and 321).
  // Of few rows it is the launches, and the form without quantizing kernels
  // (16) is shorter, three launches against five: 16 x 8 slots of 128 experts of
  // 2688 x 1856 138 us and 143, of 1088 x 896 39 and 49; 32 slots of 4 experts of
  // 512 x 512 14 and 16.5.  But there every CTA quantizes its experts' rows
  // itself, which pays up to about 16384 values an expert: 111 slots of 30
  // experts of 2688 x 1856 (16800) 76 us and 68, 64 of 4 (72700) 34 and 24.
  const int64_t mean = L.slots / experts;
  const bool few = L.slots <= kStreamSlots && L.slots * (H + I) <= 16384 * experts;
  L.nt = mean < 1 || few ? 16 : mean < 40 ? 64 : mean < 136 ? 128 : 256;
  L.maxseg = L.slots / L.nt + (experts < L.slots ? experts : L.slots);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  L.cursor = take(experts * 4);
  L.segs = take(L.maxseg * 16);
  L.nseg = take(4);
  L.nrows = take(4);
  L.pairs = take(L.slots * 4);
  L.row_w = take(L.slots * 4);
  L.xq = take(L.slots * H);
  L.xscale = take(L.slots * 4);
  L.h = take(L.slots * I * 2);
  L.hq = take(L.slots * I);
  L.hscale = take(L.slots * 4);
  L.z = take(L.slots * H * 4);
  L.total = off;
  return L;
}

int moe_check(int64_t m, int32_t topk, const tq4_1s_int8_weight* up, const tq4_1s_int8_weight* down, bool ptrs) {
  int rc = weight_ok(up, ptrs);
  if (rc) return rc;
  if ((rc = weight_ok(down, ptrs))) return rc;
  if (m < 0 || topk <= 0 || topk > 64 || m * topk > (1ll << 26)) return TQ_ERR_INVALID_ARG;
  if (up->num_experts != down->num_experts || up->k != down->n || up->n != down->k) return TQ_ERR_INVALID_ARG;
  return TQ_OK;
}

}  // namespace
}  // namespace tq4

using namespace tq4;

TQ_API int tq4_1s_int8_quantize(const void* W, int dtype, const tq4_1s_int8_weight* out, tq4_stream_t stream) {
  int rc = weight_ok(out, true);
  if (rc) return rc;
  if (!W || !dtype_ok(dtype)) return TQ_ERR_INVALID_ARG;
  if (!aligned16(W)) return TQ_ERR_ALIGNMENT;
  const int64_t rows = out->n * out->num_experts;
  if (rows > INT32_MAX) return TQ_ERR_INVALID_ARG;
  if ((rc = check_device(nullptr))) return rc;
  if (take_injected_failure()) return TQ_ERR_CUDA;
  RowsArgs a{};
  a.x = W;
  a.ldx = a.k = out->k;
  a.rows = rows;
  a.q = out->q;
  a.scale = out->wscale;
  return rc_of(launch_rows(dtype, a, reinterpret_cast<cudaStream_t>(stream)));
}

TQ_API int tq4_1s_int8_dequantize(const tq4_1s_int8_weight* w, float* W_out, tq4_stream_t stream) {
  int rc = weight_ok(w, true);
  if (rc) return rc;
  if (!W_out) return TQ_ERR_INVALID_ARG;
  if (!aligned16(W_out)) return TQ_ERR_ALIGNMENT;
  if ((rc = check_device(nullptr))) return rc;
  if (take_injected_failure()) return TQ_ERR_CUDA;
  const int64_t rows = w->n * w->num_experts, kg = w->k / 4;
  const int64_t blocks = (rows * kg + 256 * kDeqGroups - 1) / (256 * kDeqGroups);
  if (blocks > INT32_MAX) return TQ_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_early(cfg, attr, static_cast<unsigned>(blocks), 256, 0, reinterpret_cast<cudaStream_t>(stream));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, int8_dequantize_kernel, static_cast<const int8_t*>(w->q),
                                           static_cast<const float*>(w->wscale), W_out, rows, static_cast<int32_t>(kg));
  if (e != cudaSuccess) return TQ_ERR_CUDA;
  note_launches(1);
  return rc_of(cudaGetLastError());
}

TQ_API size_t tq4_1s_linear_int8_workspace(int64_t m, const tq4_1s_int8_weight* w) {
  if (m <= 0 || m > (1ll << 24) || weight_ok(w, false) != TQ_OK || w->num_experts != 1) return 0;
  if (streams(m, w->k)) return 0;
  return linear_layout(m, w->k).total;
}

TQ_API int tq4_1s_linear_int8(const void* x, int dtype, int64_t m, int64_t ldx, const tq4_1s_int8_weight* w, void* y,
                              void* ws, size_t ws_bytes, tq4_stream_t stream) {
  int rc = weight_ok(w, true);
  if (rc) return rc;
  if (w->num_experts != 1 || m < 0 || m > (1ll << 24) || !dtype_ok(dtype) || ldx < w->k || ldx > (1ll << 40))
    return TQ_ERR_INVALID_ARG;
  if (m == 0) return TQ_OK;
  if (!x || !y) return TQ_ERR_INVALID_ARG;
  if (!aligned_elem(x, dtype) || !aligned16(y)) return TQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  const Plan p = plan_dense(m, w->n, w->k, sms);
  if (p.row_tiles * p.tok_tiles > kMaxTiles) return TQ_ERR_INVALID_ARG;   // 32-bit tile numbers
  const int64_t bytes = dtype == TQ_DTYPE_F32 ? 4 : 2;
  const uintptr_t x0 = reinterpret_cast<uintptr_t>(x), y0 = reinterpret_cast<uintptr_t>(y);
  if (x0 < y0 + static_cast<uintptr_t>(m * w->n * bytes) &&
      y0 < x0 + static_cast<uintptr_t>(((m - 1) * ldx + w->k) * bytes))
    return TQ_ERR_INVALID_ARG;   // y over x: other CTAs may still read x when the first write y
  const bool stream_rows = streams(m, w->k);
  const LinearLayout L = linear_layout(m, w->k);
  if (!stream_rows && (!ws || ws_bytes < L.total)) return TQ_ERR_WORKSPACE;
  if (!aligned16(ws)) return TQ_ERR_ALIGNMENT;
  if (take_injected_failure()) return TQ_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  alignas(64) CUtensorMap tw, tx;
  if (stream_rows) {
    if (!encode_i8_map(&tw, w->q, w->num_experts, w->n, w->k, 128)) return TQ_ERR_CUDA;
    Int8StreamArgs a{};
    a.test_withhold = withhold_arrival_hook() ? 1 : 0;
    a.n = static_cast<int32_t>(w->n);
    a.k = static_cast<int32_t>(w->k);
    a.m = static_cast<int32_t>(m);
    a.row_tiles = static_cast<int32_t>(p.row_tiles);
    a.ksteps = static_cast<int32_t>(p.ksteps);
    a.mode = INT8_DENSE;
    a.dtype = dtype;
    a.parts = int8_stream_parts(p.row_tiles, p.ksteps, sms);
    a.ldx = ldx;
    a.x = x;
    a.wscale = w->wscale;
    a.y = y;
    return rc_of(launch_int8_stream(dtype, tw, a, p.row_tiles, sms, st));
  }
  uint8_t* base = static_cast<uint8_t*>(ws);
  int8_t* xq = reinterpret_cast<int8_t*>(base + L.xq);
  if (!encode_i8_map(&tw, w->q, w->num_experts, w->n, w->k, 128) ||
      !encode_i8_map(&tx, xq, 0, m, w->k, p.nt == kInt8Pair ? 128 : p.nt))
    return TQ_ERR_CUDA;
  RowsArgs r{};
  r.x = x;
  r.ldx = ldx;
  r.k = w->k;
  r.rows = m;
  r.q = xq;
  r.scale = reinterpret_cast<float*>(base + L.xscale);
  if (launch_rows(dtype, r, st) != cudaSuccess) return TQ_ERR_CUDA;
  Int8GemmArgs a{};
  a.test_withhold = withhold_arrival_hook() ? 1 : 0;
  a.n = static_cast<int32_t>(w->n);
  a.m = static_cast<int32_t>(m);
  a.row_tiles = static_cast<int32_t>(p.row_tiles);
  a.tok_tiles = static_cast<int32_t>(p.tok_tiles);
  a.ksteps = static_cast<int32_t>(p.ksteps);
  a.mode = INT8_DENSE;
  a.dtype = dtype;
  a.xscale = r.scale;
  a.wscale = w->wscale;
  a.y = y;
  return rc_of(launch_int8_gemm(tw, tx, a, p.nt, p.grid, st));
}

TQ_API size_t tq4_1s_moe_int8_workspace(int64_t m, int32_t topk, const tq4_1s_int8_weight* up,
                                        const tq4_1s_int8_weight* down) {
  if (moe_check(m, topk, up, down, false) != TQ_OK || m == 0) return 0;
  return moe_layout(m, topk, up->num_experts, up->k, up->n).total;
}

TQ_API int tq4_1s_moe_int8(const void* x, int dtype, int64_t m, const int32_t* topk_ids, const float* topk_w,
                           int32_t topk, const tq4_1s_int8_weight* up, const tq4_1s_int8_weight* down, void* y,
                           void* ws, size_t ws_bytes, tq4_stream_t stream) {
  int rc = moe_check(m, topk, up, down, true);
  if (rc) return rc;
  if (dtype != TQ_DTYPE_BF16 && dtype != TQ_DTYPE_F16) return TQ_ERR_INVALID_ARG;
  if (m == 0) return TQ_OK;
  if (!x || !y || !topk_ids || !topk_w) return TQ_ERR_INVALID_ARG;
  if (!aligned_elem(x, dtype) || !aligned16(y) || reinterpret_cast<uintptr_t>(topk_ids) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(topk_w) % 4 != 0)
    return TQ_ERR_ALIGNMENT;
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  const int64_t H = up->k, I = up->n, E = up->num_experts;
  const MoeLayout L = moe_layout(m, topk, E, H, I);
  const int64_t rt_up = (I + 127) / 128, rt_dn = (H + 127) / 128;
  if (L.maxseg * rt_up > kMaxTiles || L.maxseg * rt_dn > kMaxTiles) return TQ_ERR_INVALID_ARG;   // 32-bit tile numbers
  if (!ws || ws_bytes < L.total) return TQ_ERR_WORKSPACE;
  if (!aligned16(ws)) return TQ_ERR_ALIGNMENT;
  if (take_injected_failure()) return TQ_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  auto i32 = [&](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  auto f32 = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
  int8_t* xq = reinterpret_cast<int8_t*>(base + L.xq);
  int8_t* hq = reinterpret_cast<int8_t*>(base + L.hq);
  int4* segs = reinterpret_cast<int4*>(base + L.segs);
  // few rows an expert: the products quantize their rows themselves
  const bool stream_rows = L.nt == kStreamTokens && int8_stream_fits(H) && int8_stream_fits(I);
  alignas(64) CUtensorMap tu, tx, td, th;
  if (!encode_i8_map(&tu, up->q, E, I, H, 128) || !encode_i8_map(&td, down->q, E, H, I, 128)) return TQ_ERR_CUDA;
  if (!stream_rows && (!encode_i8_map(&tx, xq, 0, L.slots, H, L.nt) || !encode_i8_map(&th, hq, 0, L.slots, I, L.nt)))
    return TQ_ERR_CUDA;
  // and where the slots fit a block's routing they need no kernel for that
  const bool routed = stream_rows && L.slots <= kStreamSlots;
  const SegmentArgs sa{topk_ids,      L.slots, static_cast<int32_t>(E), L.nt, i32(L.cursor), segs,
                       i32(L.nseg),   i32(L.nrows)};
  RowsArgs r{};
  r.x = x;
  r.ldx = r.k = H;
  r.rows = m;
  r.q = xq;
  r.scale = f32(L.xscale);
  r.ids = topk_ids;
  r.topk = topk;
  r.num_experts = static_cast<int32_t>(E);
  r.cursor = i32(L.cursor);
  r.pairs = i32(L.pairs);
  r.topk_w = topk_w;
  r.row_w = f32(L.row_w);
  // (where the rows count their places, their kernel writes the segments too)
  const bool counted =
      !stream_rows && (dtype == TQ_DTYPE_BF16 ? rows_count<__nv_bfloat16>(r) : rows_count<__half>(r));
  if (!routed && !counted) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    launch_early(cfg, attr, 1, 1024, static_cast<size_t>(E) * 4, st);
    if (cudaLaunchKernelEx(&cfg, int8_segments_kernel, sa, topk_w,
                           stream_rows ? i32(L.pairs) : static_cast<int32_t*>(nullptr), f32(L.row_w)) != cudaSuccess)
      return TQ_ERR_CUDA;
    note_launches(1);
  }
  const int64_t tiles_up = L.maxseg * rt_up, tiles_dn = L.maxseg * rt_dn;
  if (stream_rows) {
    Int8StreamArgs s{};
    s.test_withhold = withhold_arrival_hook() ? 1 : 0;
    s.n = static_cast<int32_t>(I);
    s.k = static_cast<int32_t>(H);
    s.row_tiles = static_cast<int32_t>(rt_up);
    s.ksteps = static_cast<int32_t>((H + 127) / 128);
    s.mode = INT8_UP;
    s.parts = 1;
    s.topk = topk;
    s.ldx = H;
    s.x = x;
    if (routed) {
      s.ids = topk_ids;
      s.topk_w = topk_w;
      s.slots = static_cast<int32_t>(L.slots);
      s.experts = static_cast<int32_t>(E);
    } else {
      s.segs = segs;
      s.nseg = i32(L.nseg);
      s.pairs = i32(L.pairs);
      s.row_w = f32(L.row_w);
    }
    s.wscale = up->wscale;
    s.y = base + L.h;
    if (launch_int8_stream(dtype, tu, s, tiles_up, sms, st) != cudaSuccess) return TQ_ERR_CUDA;
    s.n = static_cast<int32_t>(H);
    s.k = static_cast<int32_t>(I);
    s.row_tiles = static_cast<int32_t>(rt_dn);
    s.ksteps = static_cast<int32_t>((I + 127) / 128);
    s.mode = INT8_DOWN;
    s.ldx = I;
    s.x = base + L.h;
    s.wscale = down->wscale;
    s.y = base + L.z;
    if (launch_int8_stream(TQ_DTYPE_BF16, td, s, tiles_dn, sms, st) != cudaSuccess) return TQ_ERR_CUDA;
  } else {
    if (launch_rows(dtype, r, st, counted ? &sa : nullptr) != cudaSuccess) return TQ_ERR_CUDA;
    Int8GemmArgs a{};
    a.test_withhold = withhold_arrival_hook() ? 1 : 0;
    a.n = static_cast<int32_t>(I);
    a.row_tiles = static_cast<int32_t>(rt_up);
    a.ksteps = static_cast<int32_t>((H + 127) / 128);
    a.mode = INT8_UP;
    a.segs = segs;
    a.nseg = i32(L.nseg);
    a.xscale = f32(L.xscale);
    a.wscale = up->wscale;
    a.y = base + L.h;
    if (launch_int8_gemm(tu, tx, a, L.nt, static_cast<int>(tiles_up < sms ? tiles_up : sms), st) != cudaSuccess)
      return TQ_ERR_CUDA;
    RowsArgs g{};
    g.x = base + L.h;
    g.ldx = g.k = I;
    g.rows = L.slots;
    g.q = hq;
    g.scale = f32(L.hscale);
    g.rows_dev = i32(L.nrows);
    if (launch_rows(TQ_DTYPE_BF16, g, st) != cudaSuccess) return TQ_ERR_CUDA;
    a.n = static_cast<int32_t>(H);
    a.row_tiles = static_cast<int32_t>(rt_dn);
    a.ksteps = static_cast<int32_t>((I + 127) / 128);
    a.mode = INT8_DOWN;
    a.xscale = f32(L.hscale);
    a.wscale = down->wscale;
    a.pairs = i32(L.pairs);
    a.row_w = f32(L.row_w);
    a.y = base + L.z;
    if (launch_int8_gemm(td, th, a, L.nt, static_cast<int>(tiles_dn < sms ? tiles_dn : sms), st) != cudaSuccess)
      return TQ_ERR_CUDA;
  }
  const int32_t hg = static_cast<int32_t>(H / 4), experts = static_cast<int32_t>(E);
  const unsigned blocks = static_cast<unsigned>((m * hg + 255) / 256);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_early(cfg, attr, blocks, 256, 0, st);
  const float* z = f32(L.z);
  const cudaError_t e =
      dtype == TQ_DTYPE_BF16
          ? cudaLaunchKernelEx(&cfg, int8_combine_kernel<__nv_bfloat16>, z, topk_ids, m, topk, hg, experts,
                               static_cast<__nv_bfloat16*>(y))
          : cudaLaunchKernelEx(&cfg, int8_combine_kernel<__half>, z, topk_ids, m, topk, hg, experts,
                               static_cast<__half*>(y));
  if (e != cudaSuccess) return TQ_ERR_CUDA;
  note_launches(1);
  return rc_of(cudaGetLastError());
}
