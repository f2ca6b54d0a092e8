// The scored expert router (tq4_1s_router_scored): softmax or sigmoid scores,
// a balance bias that takes part in the choice only, groups of experts of
// which the best are kept, top-k, renormalised and scaled weights.
//
// One warp per token; lane l holds the experts l, l + 32, ...  Scores are
// computed in fp64, so that the choice is that of the exact scores except for
// differences near 1e-16.  Without a bias the order of the scores is the order
// of the logits, and the choice is made on those.
#include "tq4_internal.h"

#define TQ_API extern "C" __attribute__((visibility("default")))

namespace tq4 {
namespace {

constexpr int kMaxExperts = 1024, kMaxTopk = 32, kMaxGroups = 32;
constexpr int kWarps = 4;

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
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// PL: experts per lane.
template <typename T, int PL>
__global__ void __launch_bounds__(kWarps * 32) router_scored_kernel(const __grid_constant__ RouterArgs a) {
  __shared__ double s_choice[kWarps][PL * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= a.m) return;
  const T* zt = static_cast<const T*>(a.logits) + t * a.experts;
  const double kInf = INFINITY;
  double score[PL], choice[PL];
  uint32_t open = 0;   // bit i: expert lane + 32 i can be chosen
  bool bad = false;
  double top = -kInf;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int e = lane + 32 * i;
    const float z = e < a.experts ? load_logit(zt + e) : -INFINITY;
    const bool number = z == z;
    if (e < a.experts && number) open |= 1u << i;
    bad |= !number;
    choice[i] = number ? static_cast<double>(z) : -kInf;
    top = fmax(top, choice[i]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PL; ++i) score[i] = ((open >> i) & 1u) ? 1.0 / (1.0 + exp(-choice[i])) : 0.0;
  } else {
    top = warp_max(top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      score[i] = top == -kInf ? 0.0 : choice[i] == top ? 1.0 : exp(choice[i] - top);
      sum += score[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < PL; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (!((open >> i) & 1u)) continue;
      const float b = __ldg(a.bias + e);
      if (!(b < INFINITY)) {   // NaN or +inf
        bad = true;
        open &= ~(1u << i);
      }
      choice[i] = score[i] + static_cast<double>(b);
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) raise_status(TQ_DEV_NONFINITE);
  if (a.keep < a.groups) {
    // lane g ranks group g
    const bool by_score = a.top2 && !a.bias;   // sums need the scores themselves
#pragma unroll
    for (int i = 0; i < PL; ++i)
      s_choice[warp][lane + 32 * i] = ((open >> i) & 1u) ? (by_score ? score[i] : choice[i]) : -kInf;
    __syncwarp();
    const int size = a.experts / a.groups;
    double first = -kInf, second = -kInf;
    if (lane < a.groups)
      for (int i = 0; i < size; ++i) {
        const double c = s_choice[warp][lane * size + i];
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
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.experts && !((kept >> (e / size)) & 1u)) open &= ~(1u << i);
    }
  }
  double mine = 0.0;   // lane j: the score of the j-th choice
  int my_id = -1;
  for (int j = 0; j < a.topk; ++j) {
    double bc = -kInf, bs = 0.0;
    int be = INT32_MAX;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (((open >> i) & 1u) && (be == INT32_MAX || choice[i] > bc)) {
        bc = choice[i];
        bs = score[i];
        be = lane + 32 * i;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double oc = __shfl_xor_sync(0xFFFFFFFFu, bc, o), os = __shfl_xor_sync(0xFFFFFFFFu, bs, o);
      const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, o);
      if (oc > bc || (oc == bc && oe < be)) {
        bc = oc;
        bs = os;
        be = oe;
      }
    }
    if (be == INT32_MAX) break;   // (the whole warp agrees)
    if ((be & 31) == lane) open &= ~(1u << (be >> 5));
    if (lane == j) {
      mine = bs;
      my_id = be;
    }
  }
  if (a.renorm) {
    const double sum = warp_sum(mine);
    mine = sum > 0.0 ? mine / sum : 0.0;
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = static_cast<float>(mine * static_cast<double>(a.scale));
  }
}

template <typename T>
cudaError_t launch_pl(const RouterArgs& a, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>((a.m + kWarps - 1) / kWarps);
  const int per = (a.experts + 31) / 32;
  if (per <= 4) router_scored_kernel<T, 4><<<grid, kWarps * 32, 0, st>>>(a);
  else if (per <= 8) router_scored_kernel<T, 8><<<grid, kWarps * 32, 0, st>>>(a);
  else if (per <= 16) router_scored_kernel<T, 16><<<grid, kWarps * 32, 0, st>>>(a);
  else router_scored_kernel<T, 32><<<grid, kWarps * 32, 0, st>>>(a);
  note_launches(1);
  return cudaGetLastError();
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
