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
// float32's error (or alike in the bits that the index leaves), the row is
// selected once more with whole keys, in float64 if they are scores, so the
// selection is that of the float64 scores for every row and the cheap
// arithmetic serves nearly all of them.
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

// Selection value of expert e; -inf where it is masked.
template <typename R>
__device__ __forceinline__ R value_at(const TopkArgs& A, const Norm<R>& n, int e, float x) {
  if (!A.bias) return (R)x;
  const float b = A.bias[e];
  if (x == -topk_inf() || !(b > -topk_inf())) return (R)-topk_inf();
  return score_of<R>(x, n, A.sigmoid) + (R)b + R(0);  // never -0
}

// The open groups: bit g * lanes_per_group for each. v: the lane's selection
// values, x its logits. L lanes take a group, each a strided part of it from
// the values in shared memory; then the group's best two meet by shuffles.
// near: whether the last open group's value is within `margin` (and 2^-20 of
// its size) of the first closed one's.
template <typename R, int NV, int VEC>
__device__ __forceinline__ unsigned open_groups(const TopkArgs& A, const R (&v)[NV], const float (&x)[NV], int lane,
                                                const Norm<R>& norm, float margin, bool& near) {
  extern __shared__ __align__(16) unsigned char topk_smem[];
  R* row = reinterpret_cast<R*>(topk_smem) + (size_t)(threadIdx.x >> 5) * A.smem_row;
  const float inf = topk_inf();
  const bool sums = A.group_top == 2;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    if (e < A.experts) {
      const R w = sums && !A.bias && x[i] != -inf ? score_of<R>(x[i], norm, A.sigmoid) : v[i];
      row[e + (int)A.by_group.div((uint32_t)e)] = w;  // a value of padding per group spreads them over the banks
    }
  }
  __syncwarp();
  const int L = A.lanes_per_group, g = lane / L;
  R b1 = (R)-inf, b2 = (R)-inf;
  if (g < A.groups)
    for (int j = lane % L; j < A.group_size; j += L) {
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
  const R val = b1 + (sums && b2 > (R)-inf ? b2 : R(0));
  int ahead = 0;
  for (int h = 0; h < A.groups; h++) {
    const R o = __shfl_sync(kFull, val, h * L);
    ahead += (o > val || (o == val && h < g)) ? 1 : 0;
  }
  const bool in = g < A.groups && ahead < A.topk_groups;
  if (sizeof(R) == 4 && margin > 0.f && A.topk_groups < A.groups) {
    const uint32_t k = key_of((float)val);
    const float least = value_of(~warp_max(in ? ~k : 0u));
    const float most = value_of(warp_max(in || g >= A.groups ? kKeyNegInf : k));
    near = most > -inf && !(least - most > margin + 0x1p-20f * fmaxf(fabsf(least), fabsf(most)));
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
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    v[i] = e < A.experts ? value_at<R>(A, norm, e, x[i]) : (R)-topk_inf();
  }
  K key[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) key[i] = expert_at<VEC>(i, lane) < A.experts ? key_of(v[i]) : K(0);
  if (A.groups > 1) {
    bool near = false;
    const unsigned open = open_groups<R, NV, VEC>(A, v, x, lane, norm, 0.f, near);
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

template <int NV, int VEC, bool BF16>
__global__ void __launch_bounds__(kTopkWarps * 32, NV <= 8 ? 4 : NV == 16 ? 2 : 1) k_topk(const __grid_constant__ TopkArgs A) {
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kTopkWarps + (threadIdx.x >> 5);
  if (t >= A.T) return;
  const char* logits = static_cast<const char*>(A.logits) + t * A.stride * (BF16 ? 2 : 4);
  const float inf = topk_inf();
  float x[NV];
#pragma unroll
  for (int c = 0; c < NV / VEC; c++) {
    const int e0 = expert_at<VEC>(c * VEC, lane);
    if (VEC > 1 && e0 < A.experts) {  // experts is a multiple of VEC here, rows 16-byte aligned
      const uint4 q = ld_u4(logits + (size_t)e0 * (BF16 ? 2 : 4));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < VEC; j++) {
        const uint32_t u = w[(BF16 ? j / 2 : j) & 3];
        x[c * VEC + j] = clean(__uint_as_float(!BF16 ? u : (j & 1) ? (u & 0xffff0000u) : (u << 16)));
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j++)
        x[c * VEC + j] = e0 + j < A.experts ? clean(logit_at<BF16>(logits, e0 + j)) : -inf;
    }
  }
  // softmax needs the row's maximum, and its sum where scores themselves count
  const bool scored = A.bias != nullptr;
  const bool scores = scored || (A.groups > 1 && A.group_top == 2);
  const bool sum = !A.sigmoid && (scores || !A.renorm);
  float most = 0.f;
  if (sum) {
    most = x[0];
#pragma unroll
    for (int i = 1; i < NV; i++) most = fmaxf(most, x[i]);
    most = value_of(warp_max(key_of(most)));
  }
  const Norm<float> norm = norm_of<float, NV>(x, most, sum);
  // Bound of float32's error in a score: a few ulp of the largest one, plus
  // 2^-24 for each of the NV + 5 additions of a softmax sum; for a sigmoid
  // s (1 - s) 2^-22 from the exponential and 2^-23 from sum and quotient.
  const float eps = !scores ? 0.f : A.sigmoid ? 0x1p-22f : (NV + 16) * 0x1p-24f / fmaxf(norm.total, 1.f);

  // Packed keys: the leading bits of the value's key, then the index, inverted
  // so that ties go to the lowest. bf16 logits fit whole; of a float32 value
  // the bits that give way to the index are lost, and neighbours that then
  // look alike (or lie within the scores' error) send the row to select_row.
  constexpr uint32_t kMask = 32u * NV - 1;
  const bool whole = BF16 && !scored;
  const uint32_t cut = whole ? 0xffffu : kMask;
  uint32_t key[NV];
  bool near = false;
  {
    float v[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e = expert_at<VEC>(i, lane);
      v[i] = scored && e < A.experts ? value_at<float>(A, norm, e, x[i]) : x[i];
      key[i] = e < A.experts ? (key_of(v[i]) & ~cut) | (kMask - (uint32_t)e) : 0u;
    }
    if (A.groups > 1) {
      const unsigned open = open_groups<float, NV, VEC>(A, v, x, lane, norm, 4.f * eps, near);
      close_groups<NV, VEC>(A, open, lane, key);
    }
  }
  // Each lane keeps its two best; a maximum over the warp takes one expert.
  uint32_t h1 = 0, h2 = 0;
  auto two_below = [&](uint32_t bound) {
    h1 = 0;
    h2 = 0;
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const uint32_t k = key[i] < bound ? key[i] : 0u;
      h2 = max(h2, min(h1, k));
      h1 = max(h1, k);
    }
  };
  two_below(0xffffffffu);
  uint32_t got = 0;
  const int rounds = whole ? A.topk : A.topk + 1;  // the best one left out, too
  for (int j = 0; j < rounds; j++) {
    const uint32_t top = warp_max(h1);
    if (lane == j) got = top;
    const bool mine = h1 == top;
    if (mine) {
      h1 = h2;
      h2 = 0;
    }
    if (NV > 2 && __any_sync(kFull, mine && h1 == 0 && top != 0)) {
      if (mine) two_below(top);
    }
  }
  if (!whole) {
    const uint32_t next = __shfl_down_sync(kFull, got, 1);
    // masked values share one key and are in order; so is the end of the open experts
    if (lane < A.topk && (next & ~cut) != (kKeyNegInf & ~cut) && next != 0) {
      if (!scored) {
        near = near || (got & ~cut) == (next & ~cut);
      } else {
        const float lo = value_of(got & ~cut), hi = value_of(next | cut);
        near = near || !(lo - hi > 2.f * (eps + 0x1p-23f * fmaxf(fabsf(lo), fabsf(hi))));
      }
    }
  }
  int mine = (int)(kMask - (got & cut));
  if (__any_sync(kFull, near))
    mine = scores ? select_row<double, NV, VEC, BF16>(A, logits, lane, most)
                  : select_row<float, NV, VEC, BF16>(A, logits, lane, most);

  // weights: lane j has expert j
  const bool have = lane < A.topk;
  float xm = have ? clean(logit_at<BF16>(logits, mine)) : -inf;
  if (have && scored && !(A.bias[mine] > -inf)) xm = -inf;
  float w;
  if (!A.renorm) {
    w = score_of<float>(xm, norm, A.sigmoid);
  } else {
    // relative to the largest selected logit, so that small scores keep their ratios
    const float ms = value_of(warp_max(key_of(xm)));
    if (xm == -inf)
      w = 0.f;
    else if (!A.sigmoid)
      w = xm == ms ? 1.f : expf(xm - ms);
    else
      w = xm >= 0.f ? 1.f / (1.f + expf(-xm)) : expf(xm - fminf(ms, 0.f)) / (1.f + expf(xm));
    const float total = warp_sum(w);
    w = total > 0.f ? w / total : 0.f;
  }
  if (have) {
    A.ids[t * A.topk + lane] = mine;
    A.p[t * A.topk + lane] = w * A.scale;
  }
}

template <int NV>
int launch_nv(const TopkArgs& a, int vec, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + kTopkWarps - 1) / kTopkWarps));
  cfg.blockDim = dim3(kTopkWarps * 32);
  cfg.dynamicSmemBytes = a.groups > 1 ? (size_t)kTopkWarps * a.smem_row * 8 : 0;
  cfg.stream = st;
  cudaLaunchAttribute at[1] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  constexpr int V8 = NV >= 8 ? 8 : 1, V4 = NV >= 4 ? 4 : 1;
  auto kern = bf16 ? (vec == 8 ? k_topk<NV, V8, true> : k_topk<NV, 1, true>)
                   : (vec == 4 ? k_topk<NV, V4, false> : k_topk<NV, 1, false>);
  if (cfg.dynamicSmemBytes > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) != cudaSuccess)
    return -4;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? 0 : -4;
}

}  // namespace

int launch_topk(TopkArgs a, bool bf16, cudaStream_t st) {
  a.group_size = a.experts / a.groups;
  int g2 = 1;
  while (g2 < a.groups) g2 *= 2;
  a.lanes_per_group = 32 / g2;
  a.smem_row = a.experts + a.groups;
  a.by_group = FastDiv::of((uint32_t)a.group_size);
  const int item = bf16 ? 2 : 4, per = 16 / item;
  const bool wide = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.stride % per == 0 && a.experts % per == 0;
  int nv = 1;
  while (nv * 32 < a.experts) nv *= 2;
  const int vec = wide && nv >= per ? per : 1;
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
