// The scored expert router (tq4_1s_router_scored): softmax or sigmoid scores,
// a balance bias that takes part in the choice only, groups of experts of
// which the best are kept, top-k, renormalised and scaled weights.
//
// One warp per token; lane l holds the experts l, l + 32, ...  The choice is
// that of fp64 scores, but nearly every row is decided in fp32 (see
// fast_row): errors of the fp32 scores are bounded, and only where two experts
// or groups that the choice turns on lie closer than that bound is the row
// done again in fp64 (slow_row).  fp64 scores for every expert took 251 us
// for 65536 tokens x 256 experts, at 64 fp64 lanes an SM.
#include "tq4_internal.h"

#define TQ_API extern "C" __attribute__((visibility("default")))

namespace tq4 {
namespace {

constexpr int kMaxExperts = 1024, kMaxTopk = 32, kMaxGroups = 32;
constexpr int kWarps = 4;
constexpr int32_t kNone = INT32_MIN;   // key of an expert that cannot be chosen

struct RouterArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t m;
  int32_t experts, topk, sigmoid, groups, keep, top2, renorm;
  float scale;
};

__device__ __forceinline__ float load_logit(const float* z) { return __ldg(z); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* z) {
  return bf16_bits_to_f32(__ldg(reinterpret_cast<const uint16_t*>(z)));
}

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Floats as integers of the same order, and back.
__device__ __forceinline__ int32_t key_of(float v) {
  const int32_t b = __float_as_int(v);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int32_t k) { return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF)); }

// The definition, in fp64: NaN, infinities, rows of far values and near ties.
// `choice`: the warp's shared memory, one value per expert.
template <typename T>
__device__ __noinline__ void slow_row(const RouterArgs& a, int64_t t, double* choice) {
  const int lane = threadIdx.x & 31;
  const T* zt = static_cast<const T*>(a.logits) + t * a.experts;
  const double kInf = INFINITY;
  const int per = (a.experts + 31) / 32;
  uint32_t open = 0;   // bit i: expert lane + 32 i can be chosen
  bool bad = false;
  double top = -kInf, sum = 0.0;
  for (int i = 0; i < per; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.experts) break;
    const float z = load_logit(zt + e);
    if (z == z) {
      open |= 1u << i;
      top = fmax(top, static_cast<double>(z));
    } else {
      bad = true;
    }
  }
  top = warp_max(top);
  // exp(z - max z) of softmax; the score itself of sigmoid
  auto part = [&](int e) {
    const double z = static_cast<double>(load_logit(zt + e));
    if (a.sigmoid) return 1.0 / (1.0 + exp(-z));
    return top == -kInf ? 0.0 : z == top ? 1.0 : exp(z - top);
  };
  if (!a.sigmoid) {
    for (int i = 0; i < per; ++i)
      if ((open >> i) & 1u) sum += part(lane + 32 * i);
    sum = warp_sum(sum);
  }
  auto score = [&](int e) { return a.sigmoid ? part(e) : sum > 0.0 ? part(e) / sum : 0.0; };
  const bool grouped = a.keep < a.groups;
  const bool by_score = grouped && a.top2 && !a.bias;   // sums need the scores themselves
  for (int i = 0; i < per; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.experts) break;
    double c = -kInf;
    if ((open >> i) & 1u) {
      if (a.bias) {
        const float b = __ldg(a.bias + e);
        if (b < INFINITY) {
          c = score(e) + static_cast<double>(b);
        } else {   // NaN or +inf
          bad = true;
          open &= ~(1u << i);
        }
      } else {
        c = by_score ? score(e) : static_cast<double>(load_logit(zt + e));
      }
    }
    choice[e] = c;
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) raise_status(TQ_DEV_NONFINITE);
  if (grouped) {
    __syncwarp();
    const int size = a.experts / a.groups;
    double first = -kInf, second = -kInf;   // lane g ranks group g
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double c = choice[lane * size + i];
        second = fmax(second, fmin(first, c));
        first = fmax(first, c);
      }
    const double rank = a.top2 ? first + second : first;
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double other = __shfl_sync(0xFFFFFFFFu, rank, g);
      better += (other > rank || (other == rank && g < lane)) ? 1 : 0;
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, lane < a.groups && better < a.keep);
    __syncwarp();
    for (int i = 0; i < per; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.experts) break;
      if (!((kept >> (e / size)) & 1u)) open &= ~(1u << i);
      if (by_score) choice[e] = static_cast<double>(load_logit(zt + e));
    }
  }
  int my_id = -1;   // lane j: the j-th choice
  for (int j = 0; j < a.topk; ++j) {
    double bc = -kInf;
    int be = INT32_MAX;
    for (int i = 0; i < per; ++i)
      if (((open >> i) & 1u) && (be == INT32_MAX || choice[lane + 32 * i] > bc)) {
        be = lane + 32 * i;
        bc = choice[be];
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double oc = __shfl_xor_sync(0xFFFFFFFFu, bc, o);
      const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, o);
      if (oe != INT32_MAX && (be == INT32_MAX || oc > bc || (oc == bc && oe < be))) {
        bc = oc;
        be = oe;
      }
    }
    if (be == INT32_MAX) break;   // (the whole warp agrees)
    if ((be & 31) == lane) open &= ~(1u << (be >> 5));
    if (lane == j) my_id = be;
  }
  double mine = my_id >= 0 ? score(my_id) : 0.0;
  if (a.renorm) {
    const double total = warp_sum(mine);
    mine = total > 0.0 ? mine / total : 0.0;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = static_cast<float>(mine * static_cast<double>(a.scale));
  }
  __syncwarp();
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// What a warp keeps from row to row.
template <int PL>
struct Lane {
  float bias[PL];
  uint32_t group[(PL + 3) / 4];   // the experts' groups, a byte each
  int shift;                      // 2^shift lanes rank a group
  int size, pad;                  // experts of a group, and floats between two groups' values
  bool plain;                     // every bias is finite
  __device__ __forceinline__ uint32_t group_of(int i) const { return (group[i >> 2] >> (8 * (i & 3))) & 255u; }
};

// A row in fp32; false where it has to be done by slow_row.
//
// Each expert's choice value becomes an integer of the same order whose lowest
// bits are replaced by PL - 1 - i: keys of a lane are then all different, equal
// values go to the lower i, and (as the warp takes the lowest lane of equal
// keys) to the lower id.  Each lane keeps its two largest keys; a round takes
// the largest of the warp and its lane moves on.  The topk + 1 keys taken are
// in order unless two neighbours are closer than the errors below.
//   Errors of a value c = s + b against fp64: ex2.approx and rcp.approx 2^-22
//   and 2^-23 relative, the exponent's rounding |x| 2^-23 in x e^-x terms, the
//   add of 1: under 5e-7 for sigmoid.  Softmax has the sum's roundings too,
//   PL + 5 adds: under (PL + 16) 2^-24.  The bias' add: 2^-24 |c|; the key's
//   lowest bits: PL 2^-23 |c|.
// Without a bias the keys are the logits' own, and only the lowest bits go.
template <typename T, int PL, bool SIGMOID, bool BIASED>
__device__ __forceinline__ bool fast_row(const RouterArgs& a, int64_t t, const Lane<PL>& l, float* s_value) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  constexpr float kErr = SIGMOID ? 5e-7f : (PL + 16) * 0x1p-24f;
  const int lane = threadIdx.x & 31;
  const T* zt = static_cast<const T*>(a.logits) + t * a.experts;
  const bool grouped = a.keep < a.groups;
  float v[PL];
  bool near_zero = l.plain;
#pragma unroll
  for (int i = 0; i < PL; ++i) v[i] = lane + 32 * i < a.experts ? load_logit(zt + lane + 32 * i) : 0.0f;
#pragma unroll
  for (int i = 0; i < PL; ++i) near_zero = near_zero && fabsf(v[i]) < 40.0f;   // (not of a NaN)
  // beyond 40 an fp32 weight may underflow where its fp64 form does not
  if (!__all_sync(kAll, near_zero)) return false;
  float top2 = 0.0f, sum = 1.0f;   // softmax: log2(e) times the largest logit
  if (!SIGMOID) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PL; ++i) top = fmaxf(top, lane + 32 * i < a.experts ? v[i] : -INFINITY);
    top2 = value_of(__reduce_max_sync(kAll, key_of(top))) * kLog2e;
    if (BIASED || !a.renorm || (grouped && a.top2)) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i < a.experts) sum += ex2(fmaf(v[i], kLog2e, -top2));
      sum = warp_sum(sum);
    }
  }
  const float inv = rcp(sum);
  auto score = [&](float z) { return SIGMOID ? rcp(1.0f + ex2(z * -kLog2e)) : ex2(fmaf(z, kLog2e, -top2)) * inv; };
  if (BIASED) {
#pragma unroll
    for (int i = 0; i < PL; ++i) v[i] = score(v[i]) + l.bias[i];
  }
  uint32_t kept = kAll;
  if (grouped) {
    // the values through shared memory, a group to 2^shift lanes
    const bool by_score = a.top2 && !BIASED;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.experts) s_value[e + l.group_of(i) * l.pad] = by_score ? score(v[i]) : v[i];
    }
    __syncwarp();
    const int g = lane >> l.shift, step = 1 << l.shift;
    float first = -INFINITY, second = -INFINITY;
    if (g < a.groups) {
      const float* mine = s_value + g * (l.size + l.pad);
#pragma unroll 4
      for (int i = lane & (step - 1); i < l.size; i += step) {
        const float c = mine[i];
        second = fmaxf(second, fminf(first, c));
        first = fmaxf(first, c);
      }
    }
    for (int o = step >> 1; o > 0; o >>= 1) {
      const float f = __shfl_xor_sync(kAll, first, o), s = __shfl_xor_sync(kAll, second, o);
      second = fmaxf(fminf(first, f), fmaxf(second, s));
      first = fmaxf(first, f);
    }
    const float rank = a.top2 ? first + second : first;
    int32_t key = g < a.groups ? key_of(rank) : kNone;
    int32_t last = 0;
    kept = 0;
    for (int r = 0; r < a.keep; ++r) {
      last = __reduce_max_sync(kAll, key);
      const int w = (__ffs(__ballot_sync(kAll, key == last)) - 1) >> l.shift;   // equal ranks: the lower group
      kept |= 1u << w;
      if (g == w) key = kNone;
    }
    if (BIASED || a.top2) {
      const float in = value_of(last), out = value_of(__reduce_max_sync(kAll, key));
      // two values in each rank, and the rounding of their sums
      if (in - out <= 4.0f * kErr + 0x1p-21f * fmaxf(fabsf(in), fabsf(out))) return false;
    }
    __syncwarp();   // (the next row writes s_value again)
  }
  int32_t first = kNone, second = kNone;
  int32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    key[i] = (key_of(v[i]) & ~(PL - 1)) | (PL - 1 - i);
    if (lane + 32 * i >= a.experts || !((kept >> l.group_of(i)) & 1u)) key[i] = kNone;
    second = max(second, min(first, key[i]));
    first = max(first, key[i]);
  }
  int32_t taken = kNone;   // lane j: the j-th key and its lane
  int from = 0;
  bool one_left = true;    // `second` is the lane's next key
#pragma unroll 1
  for (int j = 0; j <= a.topk; ++j) {
    const int32_t best = __reduce_max_sync(kAll, first);
    const int w = __ffs(__ballot_sync(kAll, first == best)) - 1;
    if (lane == j) {
      taken = best;
      from = w;
    }
    if (lane == w) {
      first = second;
      second = kNone;
      if (!one_left) {   // the rest of this lane's keys: those below
        first = kNone;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          const int32_t k = key[i] < best ? key[i] : kNone;
          second = max(second, min(first, k));
          first = max(first, k);
        }
      }
      one_left = !one_left;
    }
  }
  const bool got = lane <= a.topk && taken != kNone;
  const int id = from + 32 * (PL - 1 - (taken & (PL - 1)));
  const float z = got ? load_logit(zt + id) : 0.0f;
  {
    const float b = got && BIASED ? __ldg(a.bias + id) : 0.0f;
    const float mine = value_of(taken & ~(PL - 1)), next = __shfl_down_sync(kAll, mine, 1);
    const int32_t next_key = __shfl_down_sync(kAll, taken, 1);
    const float room = BIASED ? 2.0f * kErr + fmaxf(fabsf(mine), fabsf(next)) * ((PL + 2) * 0x1p-23f) : 0.0f;
    bool near = lane < a.topk && next_key != kNone && mine - next <= room;
    if (__any_sync(kAll, near)) {   // near, but not the same
      const float nz = __shfl_down_sync(kAll, z, 1), nb = __shfl_down_sync(kAll, b, 1);
      near = near && !(z == nz && b == nb);
      if (__any_sync(kAll, near)) return false;
    }
  }
  float s = 0.0f;
  if (got && lane < a.topk) {
    if (SIGMOID) s = rcp(1.0f + expf(-z));
    else s = ex2(fmaf(z, kLog2e, -top2)) * inv;
  }
  if (a.renorm) s *= rcp(warp_sum(s));
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = got ? id : -1;
    a.weights[t * a.topk + lane] = s * a.scale;
  }
  return true;
}

// PL: experts per lane (a power of two).
template <typename T, int PL, bool SIGMOID, bool BIASED>
__global__ void __launch_bounds__(kWarps * 32, PL <= 8 ? 8 : PL == 16 ? 6 : 4)
    router_scored_kernel(const __grid_constant__ RouterArgs a) {
  // a double per expert, or a float per expert and up to 31 between two groups
  constexpr int kSpace = PL * 64 > PL * 32 + 1024 ? PL * 64 : PL * 32 + 1024;
  __shared__ alignas(8) float s_space[kWarps][kSpace];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Lane<PL> l;
  bool plain = true;
#pragma unroll
  for (int i = 0; i < (PL + 3) / 4; ++i) l.group[i] = 0;
  l.size = a.experts / a.groups;
  l.shift = 0;
  while ((a.groups << (l.shift + 1)) <= 32) ++l.shift;
  l.pad = ((1 << l.shift) - l.size) & 31;   // a group's first values then lie 2^shift banks after the last group's
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    l.bias[i] = BIASED && e < a.experts ? __ldg(a.bias + e) : 0.0f;
    plain = plain && fabsf(l.bias[i]) < INFINITY;
    if (a.keep < a.groups && e < a.experts) l.group[i >> 2] |= static_cast<uint32_t>(e / l.size) << (8 * (i & 3));
  }
  l.plain = __all_sync(0xFFFFFFFFu, plain);
  // topk + 1 keys are taken, one per lane
  const bool fits = a.topk < 32;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.m; t += static_cast<int64_t>(gridDim.x) * kWarps)
    if (!fits || !fast_row<T, PL, SIGMOID, BIASED>(a, t, l, s_space[warp])) {
      __syncwarp();
      slow_row<T>(a, t, reinterpret_cast<double*>(s_space[warp]));
    }
}

template <typename T, int PL>
cudaError_t launch_as(const RouterArgs& a, cudaStream_t st) {
  // a few rows a warp: each loads the biases once
  const int64_t blocks = (a.m + kWarps - 1) / kWarps, most = 148 * 8 * 2;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  if (a.sigmoid) {
    if (a.bias) router_scored_kernel<T, PL, true, true><<<grid, kWarps * 32, 0, st>>>(a);
    else router_scored_kernel<T, PL, true, false><<<grid, kWarps * 32, 0, st>>>(a);
  } else {
    if (a.bias) router_scored_kernel<T, PL, false, true><<<grid, kWarps * 32, 0, st>>>(a);
    else router_scored_kernel<T, PL, false, false><<<grid, kWarps * 32, 0, st>>>(a);
  }
  note_launches(1);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_pl(const RouterArgs& a, cudaStream_t st) {
  const int per = (a.experts + 31) / 32;
  if (per <= 4) return launch_as<T, 4>(a, st);
  if (per <= 8) return launch_as<T, 8>(a, st);
  if (per <= 16) return launch_as<T, 16>(a, st);
  return launch_as<T, 32>(a, st);
}

}  // namespace
}  // namespace tq4

using namespace tq4;

TQ_API int tq4_1s_router_scored(const void* logits, int dtype, int64_t m, const tq4_1s_router* r, const float* bias,
                                int32_t* ids, float* weights, tq4_stream_t stream) {
  if (!r || (dtype != TQ_DTYPE_F32 && dtype != TQ_DTYPE_BF16) || m < 0) return TQ_ERR_INVALID_ARG;
  if (r->num_experts <= 0 || r->num_experts > kMaxExperts || r->topk <= 0 || r->topk > kMaxTopk ||
      r->num_groups <= 0 || r->num_groups > kMaxGroups || r->num_experts % r->num_groups != 0 ||
      r->topk_groups <= 0 || r->topk_groups > r->num_groups ||
      r->topk > r->topk_groups * (r->num_experts / r->num_groups))
    return TQ_ERR_INVALID_ARG;
  if ((r->score != TQ_SCORE_SOFTMAX && r->score != TQ_SCORE_SIGMOID) ||
      (r->group_score != TQ_GROUP_MAX && r->group_score != TQ_GROUP_TOP2) || (r->renormalize & ~1) != 0 ||
      !(r->scale > -INFINITY && r->scale < INFINITY))
    return TQ_ERR_INVALID_ARG;
  if (r->group_score == TQ_GROUP_TOP2 && r->topk_groups < r->num_groups && r->num_experts / r->num_groups < 2)
    return TQ_ERR_INVALID_ARG;   // a group of one has no second best
  if (m > (1ll << 32)) return TQ_ERR_INVALID_ARG;
  if (m == 0) return TQ_OK;
  if (!logits || !ids || !weights) return TQ_ERR_INVALID_ARG;
  const uintptr_t la = reinterpret_cast<uintptr_t>(logits);
  if (la % (dtype == TQ_DTYPE_F32 ? 4 : 2) != 0 || reinterpret_cast<uintptr_t>(bias) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(ids) % 4 != 0 || reinterpret_cast<uintptr_t>(weights) % 4 != 0)
    return TQ_ERR_ALIGNMENT;
  int rc = check_device(nullptr);
  if (rc) return rc;
  if (take_injected_failure()) return TQ_ERR_CUDA;
  RouterArgs a{logits, bias,    ids,          weights,        m,
               r->num_experts,  r->topk,      r->score == TQ_SCORE_SIGMOID ? 1 : 0,
               r->num_groups,   r->topk_groups, r->group_score == TQ_GROUP_TOP2 ? 1 : 0,
               r->renormalize,  r->scale};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TQ_DTYPE_F32 ? launch_pl<float>(a, st) : launch_pl<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
