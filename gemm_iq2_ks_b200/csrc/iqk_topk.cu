// Routing: router logits to the experts of each token and their weights.
//
// With x the row's logits and s its scores (softmax over all experts, or the
// sigmoid of each), an expert's selection value is x itself (scores keep the
// logits' order) or s + bias. Groups rank by their best value (or the sum of
// their two best); the topk best experts of the open groups are selected, ties
// to the lowest index. Masked experts (a logit or bias of -inf or NaN) come
// last and get no weight.
//
// One warp takes one token: lane l holds NV of the row's values in registers,
// and each selected expert is one warp maximum over order-preserving integer
// keys that carry the index in their last bits. Values that need scores are
// formed in float32; where two of them that decide the result lie closer than
// float32's error (or alike in the bits that the index leaves), the
// candidates are ordered anew from whole values, in float64 if they are
// scores, so the selection is that of the float64 scores for every row and the
// cheap arithmetic serves nearly all of them. Instructions bound it: 280 for a
// plain row of 256 bf16 logits, most of them on the half-rate integer pipe.
// 65536 such rows take 22 us (1.7 TB/s; with one maximum for the value and one
// for the index over whole keys 51 us; of float32 logits 30 us, 2.3 TB/s), one
// row 1.8 us. 2048 rows of grouped sigmoid routing (1170 instructions a row)
// take 7 to 8 us, and 13.5 to 14.3 us where the groups of some row are in doubt
// and one warp orders the whole row in float64 (a third of random inputs). Warps
// that loop over rows with the next one fetched ahead were slower (24.7 and
// 11.4 us).
#include <algorithm>

#include "iqk_device.cuh"
#include "iqk_internal.h"

namespace iqk {

namespace {

constexpr int kTopkWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float topk_inf() { return __int_as_float(0x7f800000); }

// NaN counts as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -topk_inf()) + 0.0f; }

__device__ __forceinline__ uint32_t clean2(uint32_t pair) {  // of two bf16 values
  const __nv_bfloat162 ninf = __nv_bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
  const __nv_bfloat162 zero = __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
  const __nv_bfloat162 v = __hadd2_rn(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&pair), ninf), zero);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Order-preserving keys of clean values. 0 marks what cannot be selected (a
// closed group, past the row's end, already taken); -inf maps above it.
constexpr uint32_t kKeyNegInf = 0x007fffffu;
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const uint64_t o = __shfl_xor_sync(kFull, v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

template <typename R>
struct KeyOf;
template <>
struct KeyOf<float> {
  using type = uint32_t;
};
template <>
struct KeyOf<double> {
  using type = uint64_t;
};

__device__ __forceinline__ float exp_r(float v) { return expf(v); }
__device__ __forceinline__ double exp_r(double v) { return exp(v); }

template <bool BF16>
__device__ __forceinline__ float logit_at(const char* row, int e) {
  if (BF16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(row)[e]);
  return reinterpret_cast<const float*>(row)[e];
}

// Index of a lane's i-th value: VEC consecutive experts per lane and load.
template <int VEC>
__device__ __forceinline__ int expert_at(int i, int lane) {
  return (i / VEC) * (32 * VEC) + lane * VEC + (i % VEC);
}

// The row's scores' common terms: the largest logit and the sum of exponentials.
template <typename R>
struct Norm {
  R most, total;
};

template <typename R>
__device__ __forceinline__ R score_of(float x, const Norm<R>& n, bool sigmoid) {
  if (x == -topk_inf()) return R(0);
  const R v = (R)x;
  if (sigmoid) return v >= R(0) ? R(1) / (R(1) + exp_r(-v)) : exp_r(v) / (R(1) + exp_r(v));
  return (v == n.most ? R(1) : exp_r(v - n.most)) / n.total;
}

// The float32 score that selects: hardware exponential and reciprocal, without
// branches (score_bound below bounds its error).
__device__ __forceinline__ float quick_score(float x, const Norm<float>& n, bool sigmoid) {
  if (sigmoid) {
    const float e = __expf(-fabsf(x)), r = __fdividef(1.f, 1.f + e);
    return x >= 0.f ? r : e * r;
  }
  return (x == n.most ? 1.f : __expf(x - n.most)) * n.total;  // total: its reciprocal here
}
template <int NV>
__device__ __forceinline__ Norm<float> quick_norm(const float (&x)[NV], float most) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; i++) s += x[i] == most ? 1.f : x[i] > -topk_inf() ? __expf(x[i] - most) : 0.f;
  return {most, __fdividef(1.f, warp_sum(s))};
}
// Bounds of its error, in units u = 2^-24. __expf(y) is documented to be within
// 2 + 1.173 |y| steps of at most 2 u each; the rounding of y = x - most adds
// |y| u. So a softmax's exponential at distance d has a relative error of
// (4 + 3.35 d) u, absolute never above 4 u. In their sum the distances count by
// weight, sum p_i d_i <= ln n for n terms (the entropy's bound), so with its
// NV + 5 additions it is within (4 + 3.35 ln(32 NV) + NV + 5) u; reciprocal (2
// steps) and product add 5 u. With ln(1024) = 6.94 that makes NV + 42, of the
// largest score. A sigmoid's exponential is within 4 u absolute, 1 + e within
// 5 u, the quotient within 9 u of itself, the product with e <= 1 within 9 u.
// Rows in doubt are dear (one whose groups are takes 2048 x 256 from 8 to
// 14 us), so the bounds are no wider than that.
template <int NV>
__device__ __forceinline__ float score_bound(const Norm<float>& n, bool sigmoid) {
  return sigmoid ? 10 * 0x1p-24f : (NV + 44) * 0x1p-24f * fminf(n.total, 1.f);
}

// Selection value of an expert with logit x and bias b; -inf where it is masked.
__device__ __forceinline__ double value_of_expert(const Norm<double>& n, bool sigmoid, float x, float b) {
  if (x == -topk_inf() || !(b > -topk_inf())) return -(double)topk_inf();
  return score_of<double>(x, n, sigmoid) + (double)b + 0.0;  // never -0
}
__device__ __forceinline__ float value_of_expert(const Norm<float>& n, bool sigmoid, float x, float b) {
  const float v = quick_score(x, n, sigmoid) + b + 0.f;
  return x == -topk_inf() || !(b > -topk_inf()) ? -topk_inf() : v;
}

// A group's value from its best two selection values, and what float32
// arithmetic may have moved it by, beyond the scores' own error: half a step
// for each of the two (score + bias) and for their sum, each relative to a
// number of at most the larger one's size m, twice: 4 m 2^-24; the rounding of
// value +- slack adds 2 m 2^-24. The sum itself may be far smaller than the
// two. A sum below float32's range stays ahead of -inf.
template <typename R>
__device__ __forceinline__ R group_value(R b1, R b2, int group_top) {
  const R v = b1 + (group_top == 2 && b2 > (R)-topk_inf() ? b2 : R(0));
  return sizeof(R) == 4 && b1 > (R)-topk_inf() ? (R)fmaxf((float)v, -3.402823466e38f) : v;
}
__device__ __forceinline__ float group_slack(float b1, float b2, int group_top) {
  const float m = fmaxf(fabsf(b1), group_top == 2 && b2 > -topk_inf() ? fabsf(b2) : 0.f);
  return 6 * 0x1p-24f * fminf(m, 3.402823466e38f);
}
// Whether the last open group (lowest value `least`, less its slack) may not be
// ahead of the first closed one (`most`, its slack added).
__device__ __forceinline__ bool groups_near(float least, float most, float margin) {
  return most > -topk_inf() && !(least - most > margin);
}

// The open groups of a row: bit g * lanes_per_group for each. v: the lane's
// selection values. L lanes take a group, each a strided part of it from the
// values in shared memory; then the group's best two meet by shuffles.
// near: whether the last open group's value is within `margin` and both slacks
// of the first closed one's.
template <typename R, int NV, int VEC>
__device__ __forceinline__ unsigned open_groups(const TopkArgs& A, const R (&v)[NV], int lane, float margin, bool& near) {
  extern __shared__ __align__(16) unsigned char topk_smem[];
  // A warp's row starts at the same byte for both types (room for 8 a value):
  // the warps of a block are not in step, one may be at its float64 pass while
  // its neighbours still read float32 values.
  R* row = reinterpret_cast<R*>(topk_smem + (size_t)(threadIdx.x >> 5) * A.smem_row * sizeof(double));
  const float inf = topk_inf();
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    if (e < A.experts) row[e + (int)A.by_group.div((uint32_t)e)] = v[i];  // padded, to spread groups over the banks
  }
  __syncwarp();
  const int L = A.lanes_per_group, g = lane >> A.lanes_log2;  // L: a power of two
  R b1 = (R)-inf, b2 = (R)-inf;
  if (g < A.groups)
    for (int j = lane & (L - 1); j < A.group_size; j += L) {
      const R w = row[g * (A.group_size + 1) + j];
      const R lo = w < b1 ? w : b1;
      b1 = w < b1 ? b1 : w;
      b2 = b2 < lo ? lo : b2;
    }
  for (int d = 1; d < L; d <<= 1) {
    const R o1 = __shfl_xor_sync(kFull, b1, d), o2 = __shfl_xor_sync(kFull, b2, d);
    const R lo = b1 < o1 ? b1 : o1;
    b1 = b1 < o1 ? o1 : b1;
    b2 = b2 < o2 ? o2 : b2;
    b2 = b2 < lo ? lo : b2;
  }
  const R val = group_value(b1, b2, A.group_top);
  int ahead = 0;
  for (int h = 0; h < A.groups; h++) {
    const R o = __shfl_sync(kFull, val, h * L);
    ahead += (o > val || (o == val && h < g)) ? 1 : 0;
  }
  const bool in = g < A.groups && ahead < A.topk_groups;
  if (sizeof(R) == 4 && margin > 0.f && A.topk_groups < A.groups) {
    const float slack = group_slack((float)b1, (float)b2, A.group_top);
    const float least = value_of(~warp_max(in ? ~key_of((float)val - slack) : 0u));
    const float most = value_of(warp_max(in || g >= A.groups ? kKeyNegInf : key_of((float)val + slack)));
    near = groups_near(least, most, margin);
  }
  return __ballot_sync(kFull, in);
}

template <int NV, int VEC, typename K>
__device__ __forceinline__ void close_groups(const TopkArgs& A, unsigned open, int lane, K (&key)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    if (e < A.experts && !((open >> ((int)A.by_group.div((uint32_t)e) * A.lanes_per_group)) & 1u)) key[i] = 0;
  }
}

// The same in registers, where `seg` (a power of two) neighbouring lanes hold a
// group: closes the other groups' keys.
template <int NV, int VEC>
__device__ __forceinline__ void close_groups_in_lanes(const TopkArgs& A, const float (&v)[NV], int lane, float margin,
                                                      uint32_t (&key)[NV], bool& near) {
  constexpr int C = NV / VEC;
  const float inf = topk_inf();
  const int seg = A.seg, per = 32 >> A.seg_log2;  // groups in a chunk of 32 * VEC experts
  const int mine = lane >> A.seg_log2;
  float val[C], slack[C];
  int ahead[C];
#pragma unroll
  for (int c = 0; c < C; c++) {
    float b1 = -inf, b2 = -inf;
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      const float w = fmaxf(v[c * VEC + j], -inf);  // what is past the row's end counts as masked
      b2 = fmaxf(b2, fminf(b1, w));
      b1 = fmaxf(b1, w);
    }
    for (int d = 1; d < seg; d <<= 1) {
      const float o1 = __shfl_xor_sync(kFull, b1, d), o2 = __shfl_xor_sync(kFull, b2, d);
      b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
      b1 = fmaxf(b1, o1);
    }
    val[c] = group_value(b1, b2, A.group_top);
    slack[c] = group_slack(b1, b2, A.group_top);
    ahead[c] = 0;
  }
#pragma unroll
  for (int c2 = 0; c2 < C; c2++)
    for (int i = 0; i < per; i++) {
      const float o = __shfl_sync(kFull, val[c2], i * seg);
      const int h = c2 * per + i;
#pragma unroll
      for (int c = 0; c < C; c++)
        ahead[c] += h < A.groups && (o > val[c] || (o == val[c] && h < c * per + mine)) ? 1 : 0;
    }
  uint32_t low = 0, high = kKeyNegInf;
#pragma unroll
  for (int c = 0; c < C; c++) {
    const bool exists = c * per + mine < A.groups, in = exists && ahead[c] < A.topk_groups;
    if (in) low = max(low, ~key_of(val[c] - slack[c]));
    if (exists && !in) high = max(high, key_of(val[c] + slack[c]));
#pragma unroll
    for (int j = 0; j < VEC; j++) key[c * VEC + j] = in ? key[c * VEC + j] : 0u;
  }
  if (margin > 0.f && A.topk_groups < A.groups) {
    const float least = value_of(~warp_max(low)), most = value_of(warp_max(high));
    near = groups_near(least, most, margin);
  }
}

template <typename R, int NV>
__device__ __forceinline__ Norm<R> norm_of(const float (&x)[NV], float most, bool need) {
  Norm<R> n{(R)most, R(1)};
  if (need) {
    R s = R(0);
#pragma unroll
    for (int i = 0; i < NV; i++)
      if (x[i] > -topk_inf()) s += x[i] == most ? R(1) : exp_r((R)x[i] - (R)most);
    n.total = warp_sum(s);
  }
  return n;
}

// The row's selection with whole keys, one warp maximum for the value and one
// minimum for the index of each expert: R = double where values are scores.
template <typename R, int NV, int VEC, bool BF16>
__device__ __noinline__ int select_row(const TopkArgs& A, const char* logits, int lane, float most) {
  using K = typename KeyOf<R>::type;
  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    x[i] = e < A.experts ? clean(logit_at<BF16>(logits, e)) : -topk_inf();
  }
  const Norm<R> norm = norm_of<R, NV>(x, most, sizeof(R) == 8 && !A.sigmoid);
  R v[NV];
  K key[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    v[i] = (R)x[i];
    if (A.bias && e < A.experts) v[i] = value_of_expert(norm, A.sigmoid, x[i], A.bias[e]);
    key[i] = e < A.experts ? key_of(v[i]) : K(0);
  }
  if (A.groups > 1) {
    if (A.group_top == 2 && !A.bias) {
#pragma unroll
      for (int i = 0; i < NV; i++)
        if (x[i] != -topk_inf()) v[i] = score_of<R>(x[i], norm, A.sigmoid);
    }
    bool near = false;
    const unsigned open = open_groups<R, NV, VEC>(A, v, lane, 0.f, near);
    close_groups<NV, VEC>(A, open, lane, key);
  }
  int mine = 0;
  for (int j = 0; j < A.topk; j++) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < NV; i++) best = key[i] > best ? key[i] : best;
    const K top = warp_max(best);
    uint32_t e = 0xffffffffu;
    if (best == top) {
#pragma unroll
      for (int i = NV - 1; i >= 0; i--)
        if (key[i] == top) e = (uint32_t)expert_at<VEC>(i, lane);
    }
    e = __reduce_min_sync(kFull, e);
    if (lane == j) mine = (int)e;
#pragma unroll
    for (int i = 0; i < NV; i++)
      if ((uint32_t)expert_at<VEC>(i, lane) == e) key[i] = 0;
  }
  return mine;
}

// Orders the n candidates (lane j < n has expert e, in roughly descending
// order; every expert left out is certainly behind the topk best of them):
// by exact logits, or by float32 scores if those are far enough apart, else by
// float64 ones. Returns lane j's expert for j < topk.
template <int NV, int VEC, bool BF16>
__device__ __noinline__ int order_candidates(const TopkArgs& A, const char* logits, int lane, int e, int n, float most,
                                             float total, float eps) {
  const float inf = topk_inf();
  const bool cand = lane < n;
  const float x = cand ? clean(logit_at<BF16>(logits, e)) : -inf;
  const float b = A.bias && cand ? A.bias[e] : 0.f;
  int src = 0;
  // lane r's source: the candidate with r others ahead of it
  auto place = [&](auto v) {
    int ahead = 0;
    for (int h = 0; h < n; h++) {
      const auto o = __shfl_sync(kFull, v, h);
      const int oe = __shfl_sync(kFull, e, h);
      ahead += (o > v || (o == v && oe < e)) ? 1 : 0;
    }
    for (int r = 0; r < min(n, A.topk + 1); r++) {
      const unsigned at = __ballot_sync(kFull, cand && ahead == r);
      if (lane == r) src = __ffs(at) - 1;
    }
  };
  if (!A.bias) {
    place(x);
  } else {
    const float v = cand ? value_of_expert(Norm<float>{most, total}, A.sigmoid, x, b) : -inf;
    place(v);
    const float here = __shfl_sync(kFull, v, src), next = __shfl_down_sync(kFull, here, 1);
    const bool near = lane < A.topk && lane + 1 < n && next > -inf &&
                      !(here - next > 2.f * (eps + 0x1p-23f * fmaxf(fabsf(here), fabsf(next))));
    if (__any_sync(kFull, near)) {
      Norm<double> norm{(double)most, 1.0};
      if (!A.sigmoid) {
        float xs[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
          const int j = expert_at<VEC>(i, lane);
          xs[i] = j < A.experts ? clean(logit_at<BF16>(logits, j)) : -inf;
        }
        norm = norm_of<double, NV>(xs, most, true);
      }
      place(cand ? value_of_expert(norm, A.sigmoid, x, b) : -(double)inf);
    }
  }
  return __shfl_sync(kFull, e, src);
}

// The two best of a lane's keys (BOUNDED: of those below `bound`).
template <bool BOUNDED, int NV>
__device__ __forceinline__ void two_best(const uint32_t (&key)[NV], uint32_t bound, uint32_t& h1, uint32_t& h2) {
  uint32_t a[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) a[i] = !BOUNDED || key[i] < bound ? key[i] : 0u;
  if (NV == 1) {
    h1 = a[0];
    h2 = 0;
    return;
  }
#pragma unroll
  for (int i = 0; i < NV / 2; i++) {
    b[i] = min(a[i], a[i + NV / 2]);
    a[i] = max(a[i], a[i + NV / 2]);
  }
#pragma unroll
  for (int n = NV / 4; n >= 1; n /= 2)
#pragma unroll
    for (int i = 0; i < n; i++) {
      b[i] = max(max(b[i], b[i + n]), min(a[i], a[i + n]));
      a[i] = max(a[i], a[i + n]);
    }
  h1 = a[0];
  h2 = b[0];
}

// PLAIN: no bias, no groups, renormalised weights; scores are then needed for
// the selected experts alone.
template <int NV, int VEC, bool BF16, bool PLAIN>
__global__ void __launch_bounds__(kTopkWarps * 32, NV <= 8 ? 4 : NV == 16 ? 2 : 1) k_topk(const __grid_constant__ TopkArgs A) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kTopkWarps + (threadIdx.x >> 5);
  if (t >= A.T) return;
  const char* logits = static_cast<const char*>(A.logits) + t * A.stride * (BF16 ? 2 : 4);
  const float inf = topk_inf();
  const float none = __uint_as_float(0xffffffffu);  // past the row's end: the key below all others
  float x[NV];
#pragma unroll
  for (int c = 0; c < NV / VEC; c++) {
    const int e0 = expert_at<VEC>(c * VEC, lane);
    if (VEC > 1) {  // experts is a multiple of VEC here, rows 16-byte aligned
      if (e0 < A.experts) {
        const uint4 q = ld_u4(logits + (size_t)e0 * (BF16 ? 2 : 4));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < VEC; j++) {
          if (BF16) {
            const uint32_t u = clean2(w[(j / 2) & 3]);
            x[c * VEC + j] = __uint_as_float((j & 1) ? (u & 0xffff0000u) : (u << 16));
          } else {
            x[c * VEC + j] = clean(__uint_as_float(w[j & 3]));
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j++) x[c * VEC + j] = none;
      }
    } else {
      x[c] = e0 < A.experts ? clean(logit_at<BF16>(logits, e0)) : none;
    }
  }
  // softmax needs the row's maximum, and its sum where scores themselves count
  const bool scored = !PLAIN && A.bias != nullptr;
  float bias[NV];
  if (scored) {
#pragma unroll
    for (int i = 0; i < NV; i += VEC > 1 ? 4 : 1) {
      const int e = expert_at<VEC>(i, lane);
      if constexpr (VEC > 1) {
        const uint4 q = e < A.experts ? ld_u4(A.bias + e) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; j++) bias[i + j] = __uint_as_float(w[j]);
      } else {
        bias[i] = e < A.experts ? A.bias[e] : 0.f;
      }
    }
  }
  const bool scores = !PLAIN && (scored || (A.groups > 1 && A.group_top == 2));
  const bool sum = !PLAIN && !A.sigmoid && (scores || !A.renorm);
  float most = 0.f;
  if (sum) {
    most = -inf;
#pragma unroll
    for (int i = 0; i < NV; i++) most = fmaxf(most, x[i]);  // `none` is a NaN, which fmaxf passes over
    most = value_of(warp_max(key_of(most)));
  }
  Norm<float> norm{most, 1.f};
  if (sum) norm = quick_norm<NV>(x, most);
  const float eps = scores ? score_bound<NV>(norm, A.sigmoid) : 0.f;

  // Packed keys: the leading bits of the value's key, then the index, inverted
  // so that ties go to the lowest. bf16 logits fit whole; of a float32 value
  // the bits that give way to the index are lost, and where neighbours then
  // look alike (or lie within the scores' error) the candidates are ordered
  // anew from whole values.
  constexpr uint32_t kMask = 32u * NV - 1;
  const bool whole = BF16 && !scored;
  const uint32_t cut = whole ? 0xffffu : kMask;
  uint32_t key[NV];
  bool near = false;
  if (scored) {
#pragma unroll
    for (int i = 0; i < NV; i++)
      x[i] = expert_at<VEC>(i, lane) < A.experts ? value_of_expert(norm, A.sigmoid, x[i], bias[i]) : none;
  }
#pragma unroll
  for (int i = 0; i < NV; i++) key[i] = (key_of(x[i]) & ~cut) | (kMask - (uint32_t)expert_at<VEC>(i, lane));
  if (!PLAIN && A.groups > 1) {
    if (scores && !scored) {
#pragma unroll
      for (int i = 0; i < NV; i++)
        if (x[i] != -inf) x[i] = quick_score(x[i], norm, A.sigmoid);
    }
    bool done = false;
    if constexpr (VEC > 1) {
      if (A.seg) {
        close_groups_in_lanes<NV, VEC>(A, x, lane, 4.f * eps, key, near);
        done = true;
      }
    }
    if (!done) {
      const unsigned open = open_groups<float, NV, VEC>(A, x, lane, 4.f * eps, near);
      close_groups<NV, VEC>(A, open, lane, key);
    }
  }
  // Each lane keeps its two best; a maximum over the warp takes one expert. A
  // lane whose two are taken shows kRefill, above all keys, and the warp then
  // fetches its next two.
  constexpr uint32_t kRefill = 0xffffffffu;
  uint32_t h1, h2, taken = 0, got = 0;
  two_best<false>(key, 0u, h1, h2);
  auto take = [&](int j) {
    uint32_t top = warp_max(h1);
    if (NV > 1 && top == kRefill) {
      if (h1 == kRefill) two_best<true>(key, taken, h1, h2);
      top = warp_max(h1);
    }
    if (lane == j) got = top;
    if (h1 == top) {
      h1 = h2;
      h2 = NV > 2 ? kRefill : 0u;
      taken = top;
    }
    return top;
  };
  uint32_t kth = 0;
  for (int j = 0; j < A.topk; j++) kth = take(j);
  int mine = (int)(kMask - (got & cut));
  bool whole_row = !PLAIN && near;  // the groups are in doubt
  if (!whole) {
    // Further candidates, until the next is certainly behind the last selected
    // one; masked values share one key, are in order, and nothing follows them.
    const float lo = value_of(kth & ~cut);
    int n = A.topk;
    if ((kth & ~cut) > (kKeyNegInf & ~cut)) {
      for (;;) {
        const uint32_t top = take(n & 31);
        if ((top & ~cut) <= (kKeyNegInf & ~cut)) break;
        const float hi = value_of(top | cut);
        if (!scored ? (top & ~cut) != (kth & ~cut)
                    : lo - hi > 2.f * (eps + 0x1p-23f * fmaxf(fabsf(lo), fabsf(hi))) || (lo == inf && hi < inf))
          break;
        if (++n > 31) break;
      }
    }
    whole_row = whole_row || n > 31;
    const uint32_t next = __shfl_down_sync(kFull, got, 1);
    bool alike = false;
    if (lane + 1 < n && (next & ~cut) > (kKeyNegInf & ~cut)) {
      const float l = value_of(got & ~cut), h = value_of(next | cut);
      alike = !scored ? (got & ~cut) == (next & ~cut)
                      : !(l - h > 2.f * (eps + 0x1p-23f * fmaxf(fabsf(l), fabsf(h))));
    }
    mine = (int)(kMask - (got & cut));
    if (!whole_row && __any_sync(kFull, alike))
      mine = order_candidates<NV, VEC, BF16>(A, logits, lane, mine, n, norm.most, norm.total, eps);
  }
  if (whole_row)
    mine = scores ? select_row<double, NV, VEC, BF16>(A, logits, lane, most)
                  : select_row<float, NV, VEC, BF16>(A, logits, lane, most);

  // weights: lane j has expert j
  const bool have = lane < A.topk;
  float xm = -inf;
  if (PLAIN && BF16)
    xm = have ? __uint_as_float(__float_as_uint(value_of(got)) & 0xffff0000u) : -inf;  // the key's bf16 half
  else if (have && (!scored || A.bias[mine] > -inf))
    xm = clean(logit_at<BF16>(logits, mine));
  float w;
  if (!PLAIN && !A.renorm) {
    w = xm == -inf ? 0.f
        : A.sigmoid ? score_of<float>(xm, norm, true)
                    : (xm == norm.most ? 1.f : expf(xm - norm.most)) * norm.total;
  } else {
    // relative to the largest selected logit, so that small scores keep their ratios
    const float ms = PLAIN ? __shfl_sync(kFull, xm, 0) : value_of(warp_max(key_of(xm)));
    if (!A.sigmoid)
      w = xm == ms ? 1.f : expf(xm - ms);
    else
      w = xm >= 0.f ? 1.f / (1.f + expf(-xm)) : expf(xm - fminf(ms, 0.f)) / (1.f + expf(xm));
    if (xm == -inf) w = 0.f;
    float total = w;  // of the first 16 lanes
#pragma unroll
    for (int d = 8; d; d >>= 1) total += __shfl_xor_sync(kFull, total, d);
    w = total > 0.f ? __fdividef(w, total) : 0.f;
  }
  if (have) {
    A.ids[t * A.topk + lane] = mine;
    A.p[t * A.topk + lane] = w * A.scale;
  }
}

template <int NV>
int launch_nv(const TopkArgs& a, int vec, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)a.T + kTopkWarps - 1) / kTopkWarps));
  cfg.blockDim = dim3(kTopkWarps * 32);
  cfg.dynamicSmemBytes = a.groups > 1 ? (size_t)kTopkWarps * a.smem_row * sizeof(double) : 0;
  cfg.stream = st;
  cudaLaunchAttribute at[1] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  constexpr int V8 = NV >= 8 ? 8 : 1, V4 = NV >= 4 ? 4 : 1;
  const bool plain = !a.bias && a.groups == 1 && a.renorm;
  auto kern = plain ? (bf16 ? (vec == 8 ? k_topk<NV, V8, true, true> : k_topk<NV, 1, true, true>)
                            : (vec == 4 ? k_topk<NV, V4, false, true> : k_topk<NV, 1, false, true>))
                    : (bf16 ? (vec == 8 ? k_topk<NV, V8, true, false> : k_topk<NV, 1, true, false>)
                            : (vec == 4 ? k_topk<NV, V4, false, false> : k_topk<NV, 1, false, false>));
  if (cfg.dynamicSmemBytes > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) != cudaSuccess)
    return -4;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? 0 : -4;
}

int log2_of(int n) {
  int l = 0;
  while (n >> (l + 1)) l++;
  return l;
}

}  // namespace

int launch_topk(TopkArgs a, bool bf16, cudaStream_t st) {
  a.group_size = a.experts / a.groups;
  int g2 = 1;
  while (g2 < a.groups) g2 *= 2;
  a.lanes_per_group = 32 / g2;
  a.lanes_log2 = log2_of(a.lanes_per_group);
  a.smem_row = a.experts + a.groups;
  a.by_group = FastDiv::of((uint32_t)a.group_size);
  const int item = bf16 ? 2 : 4, per = 16 / item;
  const bool wide = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.stride % per == 0 && a.experts % per == 0 &&
                    reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  int nv = 1;
  while (nv * 32 < a.experts) nv *= 2;
  const int vec = wide && nv >= per ? per : 1;
  // groups held by a power of two of neighbouring lanes
  const int seg = a.group_size / vec;
  a.seg = vec > 1 && a.group_size % vec == 0 && seg <= 32 && (seg & (seg - 1)) == 0 ? seg : 0;
  a.seg_log2 = log2_of(a.seg);
  switch (nv) {
    case 1: return launch_nv<1>(a, vec, bf16, st);
    case 2: return launch_nv<2>(a, vec, bf16, st);
    case 4: return launch_nv<4>(a, vec, bf16, st);
    case 8: return launch_nv<8>(a, vec, bf16, st);
    case 16: return launch_nv<16>(a, vec, bf16, st);
    case 32: return launch_nv<32>(a, vec, bf16, st);
  }
  return -3;
}

}  // namespace iqk
