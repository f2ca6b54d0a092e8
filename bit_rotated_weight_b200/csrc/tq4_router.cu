// The scored expert router (tq4_1s_router_scored): softmax or sigmoid scores,
// a balance bias that takes part in the choice only, groups of experts of
// which the best are kept, top-k, renormalised and scaled weights.
//
// Up to 255 tokens: a warp each, lane l with the experts l, l + 32, ...; more:
// four threads each (router_rows_kernel).  The choice is
// that of fp64 scores, but nearly every row is decided in fp32 (see
// fast_row): errors of the fp32 scores are bounded, and only where two experts
// or groups that the choice turns on lie closer than that bound is the row
// done again in fp64 (slow_row).  fp64 scores for every expert took 251 us
// for 65536 tokens x 256 experts (34 MB), at 64 fp64 lanes an SM; this takes 28
// us, bound by the integer units and the issue of about 300 instructions a token.  One token: 3 us.
// Rows with a logit beyond 40, a NaN or a bias that is not finite, and rows of
// topk 32, are fp64's; so is every row of the form of many rows where a bias
// lies outside [-2.5, 2.5] (389 us instead of 28; 255 rows with a bias of -inf
// 13.8 instead of 4.3).  topk 17 to 31 or more than 512 places of 256 rows and
// more take a warp a row: 65536 x 256 101 us at 17, 143 at 31, 511 at 32; 16384 x
// 1024 84, 98, 177 and 584 us at 8, 17, 31 and 32.
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

// (Plain loads: the kernel before may still write the logits and the biases
// when this one starts, which read-only loads do not allow.)
__device__ __forceinline__ float load_logit(const float* z) { return *z; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* z) {
  return bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(z));
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
#pragma unroll 4
  for (int i = 0; i < per; ++i) {
    const int e = lane + 32 * i;
    if (e >= a.experts) break;
    double c = -kInf;
    if ((open >> i) & 1u) {
      if (a.bias) {
        const float b = a.bias[e];
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
    int shift = 0;   // 2^shift lanes rank a group
    while ((a.groups << (shift + 1)) <= 32) ++shift;
    const int g = lane >> shift, step = 1 << shift;
    double first = -kInf, second = -kInf;
    if (g < a.groups)
      for (int i = lane & (step - 1); i < size; i += step) {
        const double c = choice[g * size + i];
        second = fmax(second, fmin(first, c));
        first = fmax(first, c);
      }
    for (int o = step >> 1; o > 0; o >>= 1) {
      const double f = __shfl_xor_sync(0xFFFFFFFFu, first, o), s = __shfl_xor_sync(0xFFFFFFFFu, second, o);
      second = fmax(fmin(first, f), fmax(second, s));
      first = fmax(first, f);
    }
    const double rank = a.top2 ? first + second : first;
    int better = 0;
    for (int o = 0; o < a.groups; ++o) {
      const double other = __shfl_sync(0xFFFFFFFFu, rank, o << shift);
      better += (other > rank || (other == rank && o < g)) ? 1 : 0;
    }
    uint32_t kept = 0;
    const uint32_t kept_lanes = __ballot_sync(0xFFFFFFFFu, g < a.groups && better < a.keep);
    for (int o = 0; o < a.groups; ++o) kept |= ((kept_lanes >> (o << shift)) & 1u) << o;
    __syncwarp();
    for (int i = 0; i < per; ++i) {
      const int e = lane + 32 * i;
      if (e >= a.experts) break;
      if (!((kept >> (e / size)) & 1u)) open &= ~(1u << i);
      if (by_score) choice[e] = static_cast<double>(load_logit(zt + e));
    }
  }
  int my_id = -1;   // lane j: the j-th choice
  double bc = -kInf;   // the lane's best
  int be = INT32_MAX;
  auto best_of_lane = [&]() {
    bc = -kInf;
    be = INT32_MAX;
#pragma unroll 4
    for (int i = 0; i < per; ++i)
      if (((open >> i) & 1u) && (be == INT32_MAX || choice[lane + 32 * i] > bc)) {
        be = lane + 32 * i;
        bc = choice[be];
      }
  };
  best_of_lane();
  for (int j = 0; j < a.topk; ++j) {
    // fp64 values as 64-bit integers of the same order (-0 as 0), the halves
    // reduced one after the other, then the lowest id
    const int64_t bits = __double_as_longlong(bc + 0.0);
    const int64_t key = bits ^ ((bits >> 63) & INT64_MAX);
    const bool has = be != INT32_MAX;
    if (!__any_sync(0xFFFFFFFFu, has)) break;
    const int32_t hi = static_cast<int32_t>(key >> 32);
    const int32_t top_hi = __reduce_max_sync(0xFFFFFFFFu, has ? hi : INT32_MIN);
    const bool in = has && hi == top_hi;
    const uint32_t top_lo = __reduce_max_sync(0xFFFFFFFFu, in ? static_cast<uint32_t>(key) : 0u);
    const int id = __reduce_min_sync(0xFFFFFFFFu, in && static_cast<uint32_t>(key) == top_lo ? be : INT32_MAX);
    if (lane == j) my_id = id;
    if ((id & 31) == lane) {
      open &= ~(1u << (id >> 5));
      best_of_lane();
    }
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

// exp(x) or 1 / (1 + exp(-x)), out of line: few rows need it, and code that
// they alone run has to be fetched first.
__device__ __noinline__ double exact_score(double x, bool sigmoid) {
  const double e = exp(sigmoid ? -x : x);
  return sigmoid ? 1.0 / (1.0 + e) : e;
}
// 1 / sum exp(z - top) in fp64 from the fp32 sum of 2^(z log2(e) - top2): without
// the rounding of top2, which all of the sum's terms share.
__device__ __forceinline__ double exact_inv(float top, float top2, float inv) {
  const double shared = static_cast<double>(top) * static_cast<double>(kLog2e) - static_cast<double>(top2);
  return static_cast<double>(inv) * (1.0 + 0.6931471805599453 * shared);
}
// An expert's choice value in fp64, and the part of it that the fp32 sum of
// softmax leaves uncertain: of two values that are near, the error is that of
// the difference of their parts.
struct Choice {
  double value, part;
};
template <bool SIGMOID, bool BIASED>
__device__ __forceinline__ Choice exact_choice(float z, float b, float top, double inv) {
  if (!BIASED) return {static_cast<double>(z), 0.0};
  if (SIGMOID) return {exact_score(static_cast<double>(z), true) + static_cast<double>(b), 0.0};
  const double s = exact_score(static_cast<double>(z) - static_cast<double>(top), false) * inv;
  return {s + static_cast<double>(b), s};
}
__device__ __forceinline__ bool unclear(const Choice& a, const Choice& b, float rel) {
  return a.part != b.part && fabs(a.value - b.value) <= static_cast<double>(rel) * fabs(a.part - b.part);
}

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
//   Errors of a value c = s + b against fp64.  Sigmoid: rcp.approx 2^-23 s,
//   the add of 1 2^-24 s, and through s (1 - s) <= 1/4 ex2.approx's 2^-22 and
//   the exponent's roundings, |z| 2^-23 (s (1 - s) |z| <= 0.224): under 3e-7.
//   Softmax has the sum's roundings too, in units of 2^-24 of the largest score
//   (1 / sum): PL + 5 adds, ex2's 4, its arguments' (the mean of |arg| under
//   weights 2^arg is at most log2 E, so 7) and log2(e)'s 2, rcp's 2: PL + 24.
//   The bias' add: 2^-24 |c|; the key's lowest bits: PL 2^-23 |c|.
//   A weight is off by: ex2's argument, |arg| <= 116, by log2(e)'s rounding and
// its own, ln 2 116 (1.3e-8 + 2^-24) = 5.9e-6; ex2 2^-22; the sum's adds (PL + 5
// here, up to 67 in the form of many rows) 4e-6 and its terms' arguments 5e-7;
// the sum of the topk chosen, two reciprocals and three products, 10 2^-24:
// under 1.2e-5, and near 1e-7 for logits within a few units of one another.
// Without a bias the keys are the logits' own, and only the lowest bits go (a
// bf16 logit's are zeros: nothing is lost, and equal ones are in order).
template <typename T, int PL, bool SIGMOID, bool BIASED>
__device__ __forceinline__ bool fast_row(const RouterArgs& a, int64_t t, const Lane<PL>& l, float* s_value) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
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
  float top = -INFINITY, top2 = 0.0f, sum = 1.0f;   // softmax: the largest logit, times log2(e)
  if (!SIGMOID) {
#pragma unroll
    for (int i = 0; i < PL; ++i) top = fmaxf(top, lane + 32 * i < a.experts ? v[i] : -INFINITY);
    top = value_of(__reduce_max_sync(kAll, key_of(top)));
    top2 = top * kLog2e;
    if (BIASED || !a.renorm || (grouped && a.top2)) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i < a.experts) sum += ex2(fmaf(v[i], kLog2e, -top2));
      sum = warp_sum(sum);
    }
  }
  const float inv = rcp(sum);
  constexpr float kRel = (PL + 24) * 0x1p-24f;
  const float err = SIGMOID ? 3e-7f : kRel * inv;
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
    int32_t key = g < a.groups ? key_of(rank + 0.0f) : kNone;
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
      if (in - out <= 4.0f * err + 0x1p-21f * fmaxf(fabsf(in), fabsf(out))) return false;
    }
    __syncwarp();   // (the next row writes s_value again)
  }
  int32_t first = kNone, second = kNone;
  int32_t key[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    key[i] = (key_of(v[i] + 0.0f) & ~(PL - 1)) | (PL - 1 - i);   // (-0 is 0)
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
  int id = from + 32 * (PL - 1 - (taken & (PL - 1)));
  float z = got ? load_logit(zt + id) : 0.0f;
  if constexpr (BIASED || sizeof(T) == 4) {
    const float b = got && BIASED ? a.bias[id] : 0.0f;
    const float mine = value_of(taken & ~(PL - 1)), next = __shfl_down_sync(kAll, mine, 1);
    const int32_t next_key = __shfl_down_sync(kAll, taken, 1);
    auto room = [&](float x, float y) {
      return BIASED ? 2.0f * err + fmaxf(fabsf(x), fabsf(y)) * ((PL + 2) * 0x1p-23f) : 0.0f;
    };
    bool near = lane < a.topk && next_key != kNone && mine - next <= room(mine, next);
    const bool last = (__ballot_sync(kAll, near) >> (a.topk - 1)) & 1u;
    if (last) {   // the last place is in question: is it between these two?
      const int32_t rest = __reduce_max_sync(kAll, first);
      const float edge = __shfl_sync(kAll, mine, a.topk - 1), out = value_of(rest & ~(PL - 1));
      if (rest != kNone && edge - out <= room(edge, out)) return false;
    }
    if (__any_sync(kAll, near)) {   // near, but not the same
      const float nz = __shfl_down_sync(kAll, z, 1), nb = __shfl_down_sync(kAll, b, 1);
      near = near && !(z == nz && b == nb);
    }
    const uint32_t nears = __ballot_sync(kAll, near);
    if (nears) {   // the keys taken are ranked again by their values in fp64
      const Choice c = got ? exact_choice<SIGMOID, BIASED>(z, b, top, exact_inv(top, top2, inv)) : Choice{0.0, 0.0};
      const int n = a.topk + (last ? 1 : 0);
      int place = 0;
      bool open = false;
      for (int o = 0; o < n; ++o) {
        const Choice oc = {__shfl_sync(kAll, c.value, o), SIGMOID || !BIASED ? 0.0 : __shfl_sync(kAll, c.part, o)};
        const int oid = __shfl_sync(kAll, id, o);
        const bool is = __shfl_sync(kAll, static_cast<int>(got), o) != 0;
        place += is && (oc.value > c.value || (oc.value == c.value && oid < id)) ? 1 : 0;
        open = open || (got && lane < n && is && unclear(oc, c, kRel));
      }
      if (!SIGMOID && BIASED && __any_sync(kAll, open)) return false;
      if (!got || lane >= n) place = lane;
      int new_id = id;
      float new_z = z;
      for (int o = 0; o < n; ++o) {
        const int at = __shfl_sync(kAll, place, o), oid = __shfl_sync(kAll, id, o);
        const float oz = __shfl_sync(kAll, z, o);
        if (at == lane) {
          new_id = oid;
          new_z = oz;
        }
      }
      id = new_id;
      z = new_z;
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

// One row by the whole warp, out of line: by fast_row, else by slow_row.
// `space`: a double per expert and 4 KB.
template <typename T, int PL>
__device__ __forceinline__ void lane_of(const RouterArgs& a, bool biased, Lane<PL>& l) {
  const int lane = threadIdx.x & 31;
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
    l.bias[i] = biased && e < a.experts ? a.bias[e] : 0.0f;
    plain = plain && fabsf(l.bias[i]) < INFINITY;
    if (a.keep < a.groups && e < a.experts) l.group[i >> 2] |= static_cast<uint32_t>(e / l.size) << (8 * (i & 3));
  }
  l.plain = __all_sync(0xFFFFFFFFu, plain);
}
template <typename T, bool SIGMOID, bool BIASED>
__device__ __noinline__ void again_row(const RouterArgs& a, int64_t t, bool plain, double* space) {
  bool ok = false;
  if (plain) {
    if (a.experts <= 256) {
      Lane<8> l;
      lane_of<T, 8>(a, BIASED, l);
      ok = fast_row<T, 8, SIGMOID, BIASED>(a, t, l, reinterpret_cast<float*>(space));
    } else {
      Lane<16> l;
      lane_of<T, 16>(a, BIASED, l);
      ok = fast_row<T, 16, SIGMOID, BIASED>(a, t, l, reinterpret_cast<float*>(space));
    }
  }
  __syncwarp();
  if (!ok) slow_row<T>(a, t, space);
}

// ------------------------------------------------------------------ many rows
// Four threads per token, eight tokens a warp: next to no shuffles and no idle
// lanes.  The rows lie in shared memory; eight experts at a time are turned
// into keys, sorted by a network and merged into the thread's 8 or 16 largest,
// and the four threads' lists at the end.
//
// A key's lowest bits hold the expert (all ones minus it).  Above them stand
// the highest bits of a logit's own key, or, with a bias, the choice value in
// fixed point: c + 12 lies in [8, 16) for |c| < 4, so its mantissa counts
// 2^-20 (of the float's 32 bits those above are the same for all).  A float's
// own bits, cut to make room for the expert, would count 2^-15 near 1, and
// 1.5 % of the rows would be near ties; so it is 0.1 %.  Two neighbours that
// are near are told apart in fp64 in place, and so are two groups; what is left
// (three that are near) is done again by the whole warp, which costs little
// work but 10 us of fetching code that is otherwise not run.  (27447 x 148,
// softmax with a bias: 11.7 us; 24.6 with its near pairs left to the warp, 38
// by a warp a row.)
// 14 blocks of two warps an SM: 29.4 us for 65536 x 256, 30.3 for 10, 30.4 for 28
// of one warp; warps that go on to their next rows, copied meanwhile, 32.5.
constexpr int kRowsWarps = 2, kRowsBlocks = 14;
constexpr int kRowsTopk = 16;
constexpr int kRowsOf = 8;         // tokens of a warp
constexpr int kRowsPlaces = 512;   // nine bits
constexpr int kRowsLeast = 256;

__device__ __forceinline__ void order2(int32_t& a, int32_t& b) {
  const int32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Batcher's odd-even merge sort of eight, largest first (19 exchanges).
__device__ __forceinline__ void sort8(int32_t (&k)[8]) {
  order2(k[0], k[1]), order2(k[2], k[3]), order2(k[4], k[5]), order2(k[6], k[7]);
  order2(k[0], k[2]), order2(k[1], k[3]), order2(k[4], k[6]), order2(k[5], k[7]);
  order2(k[1], k[2]), order2(k[5], k[6]);
  order2(k[0], k[4]), order2(k[1], k[5]), order2(k[2], k[6]), order2(k[3], k[7]);
  order2(k[2], k[4]), order2(k[3], k[5]);
  order2(k[1], k[2]), order2(k[3], k[4]), order2(k[5], k[6]);
}
// Keeps the K largest of two sorted lists (K and N of them), sorted; `lost`: the
// largest of the rest.
template <int K, int N>
__device__ __forceinline__ void merge(int32_t (&top)[K], const int32_t (&k)[N], int32_t& lost) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    int32_t &a = top[K - N + i], &b = top[K - N + i + 1];
    lost = max(lost, max(min(a, k[N - 1 - i]), min(b, k[N - 2 - i])));
    a = max(a, k[N - 1 - i]);
    b = max(b, k[N - 2 - i]);
  }
#pragma unroll
  for (int d = K / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (!(i & d)) order2(top[i], top[i + d]);
}

// The two largest of (first, second) and eight more.
__device__ __forceinline__ void two_of_eight(const float (&v)[8], float& first, float& second) {
  float hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = fmaxf(v[2 * i], v[2 * i + 1]);
    lo[i] = fminf(v[2 * i], v[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    second = fmaxf(fmaxf(second, lo[i]), fminf(first, hi[i]));
    first = fmaxf(first, hi[i]);
  }
}

__device__ __forceinline__ void eight(const float* z, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(z), b = *reinterpret_cast<const float4*>(z + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void eight(const __nv_bfloat16* z, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(z);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ float in_shared(const float* z) { return *z; }
__device__ __forceinline__ float in_shared(const __nv_bfloat16* z) { return __bfloat162float(*z); }

// In shared memory a group has places for `wide` experts, a multiple of eight;
// those behind its `size` hold a value that is never chosen.
constexpr float kPad = -128.0f, kPadBias = -3.9f;   // (score 0; below any bias of a row done here)
struct RowsShape {
  int pieces, stride;   // 16-byte pieces of a row, and from row to row in shared memory
  int size, wide;       // experts of a group, and its places
  int bits, mask;       // the key bits that hold the place
  float per_size, per_wide;   // 1 / size, 1 / wide
  int whole;            // rows can be copied in pieces: no padding, on 16-byte boundaries
  int bias_floats, warp_bytes;
};
template <typename T>
RowsShape rows_shape(const RouterArgs& a) {
  RowsShape s;
  s.size = a.experts / a.groups;
  s.wide = (s.size + 7) & ~7;
  const int places = s.wide * a.groups;
  s.pieces = places * static_cast<int>(sizeof(T)) / 16;
  s.stride = s.pieces | 1;
  s.per_size = 1.0f / static_cast<float>(s.size);
  s.per_wide = 1.0f / static_cast<float>(s.wide);
  s.whole = s.size == s.wide && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 ? 1 : 0;
  s.bits = 0;
  while ((1 << s.bits) < places) ++s.bits;
  s.mask = (1 << s.bits) - 1;
  // groups' biases lie 4 floats further apart, so that threads at different groups read different banks
  s.bias_floats = a.bias ? places + 4 * a.groups : 0;
  // the rows and their groups' ranks; then, in the same place, what again_row needs
  const int rows = kRowsOf * (s.stride * 16 + a.groups * 4), again = (a.experts * 8 + 4096 + 15) & ~15;
  s.warp_bytes = rows > again ? rows : again;
  return s;
}

// K: the largest keys that are kept (topk and more).
template <typename T, int K, bool SIGMOID, bool BIASED>
__global__ void __launch_bounds__(kRowsWarps * 32, kRowsBlocks) router_rows_kernel(const __grid_constant__ RouterArgs a,
                                                                         const __grid_constant__ RowsShape sh) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  extern __shared__ uint4 s_rows[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 3, own = lane >> 2;
  float* s_bias = reinterpret_cast<float*>(s_rows);
  uint8_t* mine = reinterpret_cast<uint8_t*>(s_rows) + sh.bias_floats * 4 + warp * sh.warp_bytes;
  uint4* tile = reinterpret_cast<uint4*>(mine);
  float* s_rank = reinterpret_cast<float*>(mine + kRowsOf * sh.stride * 16) + own;   // [group][token]
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRowsWarps + warp) * kRowsOf;
  pdl_wait();
  const int rows = static_cast<int>(a.m - t0 < kRowsOf ? (a.m > t0 ? a.m - t0 : 0) : kRowsOf);
  auto div_size = [&](int e) { return static_cast<int>((e + 0.5f) * sh.per_size); };   // (exact: e < 512)
  auto div_wide = [&](int e) { return static_cast<int>((e + 0.5f) * sh.per_wide); };
  const int extra = sh.wide - sh.size;
  const T* from = static_cast<const T*>(a.logits) + t0 * a.experts;
  if (sh.whole) {
    int row = 0, at = lane;
    while (at >= sh.pieces) at -= sh.pieces, ++row;
#pragma unroll 4
    for (int i = lane; i < rows * sh.pieces; i += 32) {
      const uint32_t to = smem_u32(tile + row * sh.stride + at);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(reinterpret_cast<const uint4*>(from) + i)
                   : "memory");
      at += 32;
      while (at >= sh.pieces) at -= sh.pieces, ++row;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  } else if (rows > 0) {
    T* const to = reinterpret_cast<T*>(tile);
    const int step = sh.stride * (16 / static_cast<int>(sizeof(T)));
#pragma unroll 2
    for (int e = lane; e < a.experts; e += 32) {
      T v[kRowsOf];
#pragma unroll
      for (int r = 0; r < kRowsOf; ++r) v[r] = from[(r < rows ? r : 0) * a.experts + e];
      const int at = e + div_size(e) * extra;
#pragma unroll
      for (int r = 0; r < kRowsOf; ++r) to[r * step + at] = v[r];
    }
    for (int g = 0; g < a.groups; ++g)
      for (int i = lane; i < extra * kRowsOf; i += 32)
        to[(i & (kRowsOf - 1)) * step + g * sh.wide + sh.size + i / kRowsOf] = static_cast<T>(kPad);
  }
  bool plain = true;
  if (BIASED) {
    for (int e = threadIdx.x; e < a.experts; e += kRowsWarps * 32) {
      const float b = a.bias[e];
      const int g = div_size(e);
      s_bias[e + g * (extra + 4)] = b;
      plain = plain && fabsf(b) <= 2.5f;   // (for the keys' range: 1 + 3 may round to 4; NaN and infinities too)
    }
    for (int i = threadIdx.x; i < a.groups * extra; i += kRowsWarps * 32) {
      const int g = i / extra;
      s_bias[g * (sh.wide + 4) + sh.size + (i - g * extra)] = kPadBias;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  plain = __syncthreads_and(plain);
  if (rows == 0) return;
  const T* z = reinterpret_cast<const T*>(tile + own * sh.stride);
  const bool grouped = a.keep < a.groups;
  bool done = plain && own < rows;   // decided here
  float largest = -INFINITY, top2 = 0.0f, inv = 1.0f;   // (softmax)
  if (!SIGMOID) {
    for (int e = 8 * sub; e < sh.wide * a.groups; e += 32) {
      float v[8];
      eight(z + e, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) largest = fmaxf(largest, v[i]);
    }
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(kAll, largest, 2));
    top2 = largest * kLog2e;
    if (BIASED || !a.renorm || (grouped && a.top2)) {
      float sum[2] = {0.0f, 0.0f};
      for (int e = 8 * sub; e < sh.wide * a.groups; e += 32) {
        float v[8];
        eight(z + e, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i & 1] += ex2(fmaf(v[i], kLog2e, -top2));
      }
      float all = sum[0] + sum[1];
      all += __shfl_xor_sync(kAll, all, 1);
      inv = rcp(all + __shfl_xor_sync(kAll, all, 2));
    }
  }
  // (as fast_row's, with an eighth of the row and 3 adds in a sum's chain)
  const float rel = (0.125f * static_cast<float>(a.experts) + 24.0f) * 0x1p-24f, err = SIGMOID ? 3e-7f : rel * inv;
  auto score = [&](float x) { return SIGMOID ? rcp(1.0f + ex2(x * -kLog2e)) : ex2(fmaf(x, kLog2e, -top2)) * inv; };
  uint32_t kept = 0;
  float squares = 0.0f;   // of the logits seen
  if (grouped) {
    // a group to a thread, or where their number does not suit that to all
    // four (65536 x 256 in 8 groups: 30.3 us, 33.0 by all four)
    const bool alone = a.groups % 4 == 0;
    for (int g = alone ? sub : 0; g < a.groups; g += alone ? 4 : 1) {
      float first = -INFINITY, second = -INFINITY;
      for (int j = alone ? 0 : 8 * sub; j < sh.wide; j += alone ? 8 : 32) {
        float v[8];
        eight(z + g * sh.wide + j, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) squares = fmaf(v[i], v[i], squares);
        if (BIASED || a.top2) {
          float b[8];
          if (BIASED) eight(s_bias + g * (sh.wide + 4) + j, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = BIASED ? score(v[i]) + b[i] : score(v[i]);
        }
        two_of_eight(v, first, second);
      }
      if (!alone)
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          const float f = __shfl_xor_sync(kAll, first, o), s = __shfl_xor_sync(kAll, second, o);
          second = fmaxf(fminf(first, f), fmaxf(second, s));
          first = fmaxf(first, f);
        }
      if (alone || sub == 0) s_rank[g * kRowsOf] = a.top2 ? first + second : first;
    }
    __syncwarp();
    float in = INFINITY, out = -INFINITY;
    for (int g = sub; g < a.groups; g += 4) {
      const float r = s_rank[g * kRowsOf];
      int better = 0;
#pragma unroll 4
      for (int o = 0; o < a.groups; ++o) {
        const float other = s_rank[o * kRowsOf];
        better += (other > r || (other == r && o < g)) ? 1 : 0;
      }
      if (better < a.keep) {
        kept |= 1u << g;
        in = fminf(in, r);
      } else {
        out = fmaxf(out, r);
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      kept |= __shfl_xor_sync(kAll, kept, o);
      in = fminf(in, __shfl_xor_sync(kAll, in, o));
      out = fmaxf(out, __shfl_xor_sync(kAll, out, o));
    }
    if (BIASED || a.top2) {
      // two values' errors in each rank, and the rounding of their sums
      const float room = 4.0f * err + 0x1p-21f * fmaxf(fabsf(in), fabsf(out));
      const bool unsure = done && !(in - out > room);
      if (__any_sync(kAll, unsure)) {
        // the last group kept against the first left out, in fp64
        int last = -1, first = -1, many = 0;
        for (int g = 0; g < a.groups; ++g) {
          const float r = s_rank[g * kRowsOf];
          if ((kept >> g) & 1u) {
            if (r <= out + room) last = g, many += 1;
          } else if (r >= in - room) {
            first = g, many += 16;
          }
        }
        const bool here = unsure && many == 17;   // (else slow_row's)
        // of their experts only those that fp32 leaves among the best
        double rank[2] = {0.0, 0.0}, most = 0.0;   // (the largest uncertain part)
        const double inv64 = exact_inv(largest, top2, inv);
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int g = here ? (i == 0 ? last : first) : 0;
          auto choice = [&](int j) {
            const float s = score(in_shared(z + g * sh.wide + j));
            return BIASED ? s + s_bias[g * (sh.wide + 4) + j] : s;
          };
          float one = -INFINITY, two = -INFINITY;
#pragma unroll 1
          for (int j = sub; here && j < sh.size; j += 4) {
            const float c = choice(j);
            two = fmaxf(two, fminf(one, c));
            one = fmaxf(one, c);
          }
#pragma unroll 1
          for (int o = 1; o < 4; o <<= 1) {
            const float f = __shfl_xor_sync(kAll, one, o), s = __shfl_xor_sync(kAll, two, o);
            two = fmaxf(fminf(one, f), fmaxf(two, s));
            one = fmaxf(one, f);
          }
          const float least = a.top2 ? two : one, cut = least - 2.0f * err - 0x1p-21f * fabsf(least);
          double best = -INFINITY, next = -INFINITY;
#pragma unroll 1
          for (int j = sub; here && j < sh.size; j += 4) {
            if (choice(j) < cut) continue;
            const float x = in_shared(z + g * sh.wide + j);
            // (without a bias every score has the same factor, which is left out)
            const double from_top = static_cast<double>(x) - (SIGMOID ? 0.0 : static_cast<double>(largest));
            const Choice c = BIASED ? exact_choice<SIGMOID, true>(x, s_bias[g * (sh.wide + 4) + j], largest, inv64)
                                    : Choice{exact_score(from_top, SIGMOID), 0.0};
            most = fmax(most, c.part);
            next = fmax(next, fmin(best, c.value));
            best = fmax(best, c.value);
          }
#pragma unroll 1
          for (int o = 1; o < 4; o <<= 1) {
            const double f = __shfl_xor_sync(kAll, best, o), s = __shfl_xor_sync(kAll, next, o);
            next = fmax(fmin(best, f), fmax(next, s));
            best = fmax(best, f);
          }
          rank[i] = a.top2 ? best + next : best;
        }
        if (!SIGMOID && BIASED) {
          most = fmax(most, __shfl_xor_sync(kAll, most, 1));
          most = fmax(most, __shfl_xor_sync(kAll, most, 2));
          // (two values in each rank; the difference of the parts that count is at most 2 most)
          if (here && fabs(rank[1] - rank[0]) <= 2.0 * static_cast<double>(rel) * most) done = false;
        }
        if (here && (rank[1] > rank[0] || (rank[1] == rank[0] && first < last))) kept ^= 1u << last | 1u << first;
        if (unsure && !here) done = false;
      }
    }
  } else {
    kept = (a.groups == 32 ? 0u : 1u << a.groups) - 1u;
  }
  // (nine bits of expert: [16, 24), so that the key keeps its sign bit)
  const float offset = sh.bits == 9 ? 20.0f : 12.0f;
  const uint32_t unit = sh.mask + 1;   // (a multiply-add: not the integer units' work)
  auto key_at = [&](float x, float b, int e) {
    const float c = BIASED ? score(x) + b : x + 0.0f;   // (-0 is 0)
    if (BIASED) return static_cast<int32_t>(__float_as_uint(c + offset) * unit + static_cast<uint32_t>(sh.mask - e));
    return (key_of(c) & ~sh.mask) | (sh.mask - e);
  };
  int32_t top[K], lost = kNone;
  const uint32_t stay = kept;
#pragma unroll
  for (int i = 0; i < K; ++i) top[i] = kNone;
  bool empty = true;
  for (int n = 0; n < a.keep; ++n) {
    const int g = kept ? __ffs(kept) - 1 : 0;   // (a row that holds a NaN may have kept fewer; it is not done here)
    kept &= kept - 1;
    for (int j = 8 * sub; j < sh.wide; j += 32) {
      const int e = g * sh.wide + j;
      float v[8], b[8];
      eight(z + e, v);
      if (BIASED) eight(s_bias + e + 4 * g, b);
      int32_t k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!grouped) squares = fmaf(v[i], v[i], squares);
        k[i] = key_at(v[i], BIASED ? b[i] : 0.0f, e + i);
      }
      sort8(k);
      if (empty) {
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = k[i];
        empty = false;
      } else {
        merge<K, 8>(top, k, lost);
      }
    }
  }
  // Beyond 40 an fp32 weight may underflow where its fp64 form does not.  (The
  // sum of squares leaves the integer units, which bound this kernel, alone;
  // the padding's are exact in it.)
  const bool ends = ((sh.wide / 8 - 1) & 3) == sub;   // of a group's eights this thread has the last
  const int padded = extra * (!grouped ? (ends ? 1 : 0) : a.groups % 4 == 0 ? a.groups / 4 : ends ? a.groups : 0);
  if (__any_sync(kAll, !(squares < 1600.0f + kPad * kPad * static_cast<float>(padded))))
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g)
      for (int j = sub; j < sh.size; j += 4)
        done = done && fabsf(in_shared(z + g * sh.wide + j)) < 40.0f;   // (not of a NaN)
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    int32_t k[K];
#pragma unroll
    for (int i = 0; i < K; ++i) k[i] = __shfl_xor_sync(kAll, top[i], o);
    lost = max(lost, __shfl_xor_sync(kAll, lost, o));
    merge<K, K>(top, k, lost);
  }
  // thread `sub` of the four has the choices sub, sub + 4, ...
  constexpr int kOwn = K / 4;
  int id[kOwn];
  auto expert = [&](int32_t key) { return min(sh.mask - (key & sh.mask), sh.wide * a.groups - 1); };   // (its place)
  // two scores' errors and two roundings, in counts of the fixed point
  const int room = BIASED ? static_cast<int>(2.0f * err * 0x1p20f) + 3 : 0;
  auto near = [&](int32_t hi, int32_t lo) { return lo != kNone && (hi >> sh.bits) - (lo >> sh.bits) <= room; };
  bool close[kOwn];
#pragma unroll
  for (int h = 0; h < kOwn; ++h) {
    int32_t key = top[4 * h], after = top[4 * h + 1];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (sub == i) {
        key = top[4 * h + i];
        after = 4 * h + i < K - 1 ? top[4 * h + i + 1] : lost;
      }
    id[h] = expert(key);
    // (a bf16 logit's key holds all of it)
    close[h] = (BIASED || sizeof(T) == 4) && sub + 4 * h < a.topk && near(key, after);
  }
  if (BIASED || sizeof(T) == 4) {
    uint32_t pairs = 0, one = 0, two = 0;   // bit j: choices j and j + 1 of this row are near; threads with one, two
    int h = 0;                              // which of this thread's choices
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const uint32_t c = __ballot_sync(kAll, close[i] && done) >> (lane & ~3) & 15u;
      pairs |= c << (4 * i);
      two |= one & c;
      one |= c;
      if (i > 0 && (c >> sub & 1u)) h = i;
    }
    if (__any_sync(kAll, pairs != 0)) {
      // Each such pair by its values in fp64.  Left to fast_row: three in a
      // row, a last place that two others are near, and two pairs of a thread.
      int32_t edge = kNone, third = lost, next = lost;
#pragma unroll
      for (int i = 0; i < K; ++i) {
        if (i == a.topk - 1) edge = top[i];
        if (i == a.topk) next = top[i];
        if (i == a.topk + 1) third = top[i];
      }
      const bool last = (pairs >> (a.topk - 1)) & 1u;
      if (a.topk == K && __any_sync(kAll, last)) {   // the largest below `next` was not kept
        third = kNone;
        uint32_t left = stay;
#pragma unroll 1
        for (int n = 0; n < a.keep; ++n) {
          const int g = left ? __ffs(left) - 1 : 0;
          left &= left - 1;
#pragma unroll 1
          for (int j = sub; j < sh.size; j += 4) {
            const int e = g * sh.wide + j;
            const int32_t k = key_at(in_shared(z + e), BIASED ? s_bias[e + 4 * g] : 0.0f, e);
            if (k < next) third = max(third, k);
          }
        }
        third = max(third, __shfl_xor_sync(kAll, third, 1));
        third = max(third, __shfl_xor_sync(kAll, third, 2));
      }
      if ((pairs & (pairs << 1)) || two || (last && near(edge, third))) done = false;
      bool swap = false;
      if (done && ((pairs >> (sub + 4 * h)) & 1u)) {
        int32_t after = next;
#pragma unroll
        for (int i = 1; i < K; ++i)
          if (i == sub + 4 * h + 1 && i < a.topk) after = top[i];
        int chosen = id[0];
#pragma unroll
        for (int i = 1; i < kOwn; ++i)
          if (i == h) chosen = id[i];
        const int e[2] = {chosen, expert(after)};
        const double inv64 = exact_inv(largest, top2, inv);
        Choice v[2];
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
          v[i] = exact_choice<SIGMOID, BIASED>(in_shared(z + e[i]) + 0.0f,
                                               BIASED ? s_bias[e[i] + 4 * div_wide(e[i])] : 0.0f, largest, inv64);
        swap = v[1].value > v[0].value || (v[1].value == v[0].value && e[1] < e[0]);
        if (!SIGMOID && BIASED && unclear(v[0], v[1], rel)) done = false;
      }
      uint32_t swaps = 0;   // bit j: choices j and j + 1 of this row change places
#pragma unroll
      for (int i = 0; i < kOwn; ++i) swaps |= (__ballot_sync(kAll, swap && h == i) >> (lane & ~3) & 15u) << (4 * i);
#pragma unroll
      for (int g = 0; g < kOwn; ++g) {
        const int j = sub + 4 * g;
        int32_t key = kNone;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          if (i == j + 1 && i < a.topk && (swaps >> j & 1u)) key = top[i];
          if (i + 1 == j && (swaps >> i & 1u)) key = top[i];
        }
        if (j == a.topk - 1 && (swaps >> j & 1u)) key = next;
        if (key != kNone) id[g] = expert(key);
      }
    }
  }
  float w[kOwn];
#pragma unroll
  for (int h = 0; h < kOwn; ++h) {
    w[h] = 0.0f;
    if (sub + 4 * h < a.topk) {
      const float x = in_shared(z + id[h]);
      w[h] = SIGMOID ? rcp(1.0f + expf(-x)) : ex2(fmaf(x, kLog2e, -top2)) * inv;
    }
  }
  if (a.renorm) {   // summed in the order of fast_row's shuffles: the same bits
    float total;
    if constexpr (K == 16) total = (w[0] + w[2]) + (w[1] + w[3]);
    else total = w[0] + w[1];
    total += __shfl_xor_sync(kAll, total, 2);
    const float f = rcp(total + __shfl_xor_sync(kAll, total, 1));
#pragma unroll
    for (int h = 0; h < kOwn; ++h) w[h] *= f;
  }
  const uint32_t undone = __ballot_sync(kAll, !done && own < rows);   // (no thread needs the rows any more)
  const bool redo = ((undone >> (lane & ~3)) & 15u) != 0;
  if (!redo && own < rows) {
#pragma unroll
    for (int h = 0; h < kOwn; ++h)
      if (sub + 4 * h < a.topk) {
        const int64_t at = (t0 + own) * a.topk + sub + 4 * h;
        a.ids[at] = id[h] - div_wide(id[h]) * extra;
        a.weights[at] = w[h] * a.scale;
      }
  }
  for (int r = 0; undone >> (4 * r) != 0 && r < rows; ++r)
    if ((undone >> (4 * r)) & 15u)
      again_row<T, SIGMOID, BIASED>(a, t0 + r, plain, reinterpret_cast<double*>(mine));
}

// PL: experts per lane (a power of two).
template <typename T, int PL, bool SIGMOID, bool BIASED>
__global__ void __launch_bounds__(kWarps * 32, PL <= 8 ? 8 : PL == 16 ? 6 : 4)
    router_scored_kernel(const __grid_constant__ RouterArgs a) {
  // a double per expert, or a float per expert and up to 31 between two groups
  constexpr int kSpace = PL * 64 > PL * 32 + 1024 ? PL * 64 : PL * 32 + 1024;
  __shared__ alignas(8) float s_space[kWarps][kSpace];
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  Lane<PL> l;
  lane_of<T, PL>(a, BIASED, l);
  // topk + 1 keys are taken, one per lane
  const bool fits = a.topk < 32;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.m; t += stride)
    if (!fits || !fast_row<T, PL, SIGMOID, BIASED>(a, t, l, s_space[warp])) {
      __syncwarp();
      slow_row<T>(a, t, reinterpret_cast<double*>(s_space[warp]));
    }
}

// A launch that may be set up while the kernel before it still runs (the
// kernels wait for its end first).  A plain launch of one row costs the host a
// microsecond more (4.8 and 3.6 us a call), and the GPU 0.2.
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

template <typename T, int PL>
cudaError_t launch_as(const RouterArgs& a, cudaStream_t st) {
  // a few rows a warp: each loads the biases once
  const int64_t blocks = (a.m + kWarps - 1) / kWarps, most = 148 * 8 * 2;
  const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_early(cfg, attr, grid, kWarps * 32, 0, st);
  const cudaError_t e =
      a.sigmoid ? (a.bias ? cudaLaunchKernelEx(&cfg, router_scored_kernel<T, PL, true, true>, a)
                          : cudaLaunchKernelEx(&cfg, router_scored_kernel<T, PL, true, false>, a))
                : (a.bias ? cudaLaunchKernelEx(&cfg, router_scored_kernel<T, PL, false, true>, a)
                          : cudaLaunchKernelEx(&cfg, router_scored_kernel<T, PL, false, false>, a));
  if (e != cudaSuccess) return e;
  note_launches(1);
  return cudaGetLastError();
}
template <typename T>
bool rows_fit(const RouterArgs& a) {
  return a.m >= kRowsLeast && a.topk <= kRowsTopk && a.topk < a.keep * (a.experts / a.groups) &&
         (a.experts / a.groups + 7) / 8 * 8 * a.groups <= kRowsPlaces;
}
template <typename T, int K, bool SIGMOID, bool BIASED>
cudaError_t launch_rows_of(const RouterArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  const cudaError_t e = once_per_device(attr_done, [] {
    return cudaFuncSetAttribute(router_rows_kernel<T, K, SIGMOID, BIASED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                160 * 1024);
  });
  if (e != cudaSuccess) return e;
  const RowsShape s = rows_shape<T>(a);
  const int64_t rows = kRowsOf * kRowsWarps;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  launch_early(cfg, attr, static_cast<unsigned>((a.m + rows - 1) / rows), kRowsWarps * 32,
               s.bias_floats * 4 + kRowsWarps * s.warp_bytes, st);
  const cudaError_t r = cudaLaunchKernelEx(&cfg, router_rows_kernel<T, K, SIGMOID, BIASED>, a, s);
  if (r != cudaSuccess) return r;
  note_launches(1);
  return cudaGetLastError();
}

// 8 keys a thread, or 16, which cost more: 65536 x 256 28 us and 32 (a warp a row,
// topk = 9: 80).
template <typename T, bool SIGMOID, bool BIASED>
cudaError_t launch_rows(const RouterArgs& a, cudaStream_t st) {
  return a.topk <= 8 ? launch_rows_of<T, 8, SIGMOID, BIASED>(a, st) : launch_rows_of<T, 16, SIGMOID, BIASED>(a, st);
}

template <typename T>
cudaError_t launch_pl(const RouterArgs& a, cudaStream_t st) {
  if (rows_fit<T>(a)) {
    if (a.sigmoid) return a.bias ? launch_rows<T, true, true>(a, st) : launch_rows<T, true, false>(a, st);
    return a.bias ? launch_rows<T, false, true>(a, st) : launch_rows<T, false, false>(a, st);
  }
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
  const bool grouped = r->topk_groups < r->num_groups;   // (all of them kept: no groups)
  RouterArgs a{logits, bias,    ids,          weights,        m,
               r->num_experts,  r->topk,      r->score == TQ_SCORE_SIGMOID ? 1 : 0,
               grouped ? r->num_groups : 1, grouped ? r->topk_groups : 1, r->group_score == TQ_GROUP_TOP2 ? 1 : 0,
               r->renormalize,  r->scale};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == TQ_DTYPE_F32 ? launch_pl<float>(a, st) : launch_pl<__nv_bfloat16>(a, st);
  return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
