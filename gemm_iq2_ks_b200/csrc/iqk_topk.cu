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
// keys. Values that need scores are formed in float32; where two of them that
// decide the result lie closer than float32's error, the row is selected once
// more in float64, so the selection is that of the float64 scores for every
// row and the cheap arithmetic serves nearly all of them.
#include <algorithm>

#include "iqk_device.cuh"
#include "iqk_internal.h"

namespace iqk {

namespace {

constexpr int kTopkWarps = 8;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float topk_inf() { return __int_as_float(0x7f800000); }

// Order-preserving keys. 0 marks what cannot be selected (a closed group, past
// the row's end, already taken); -inf maps above it. NaN never gets here.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 and +0 tie
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double value_of(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
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

// Selects the row's experts: lane j < topk ends with expert j in `mine`.
// Returns whether float32's error leaves the selection open (R = float only).
template <typename R, int NV, int VEC, bool BF16>
__device__ __forceinline__ bool select_row(const TopkArgs& A, const char* logits, const float (&x)[NV], int lane,
                                           const Norm<R>& norm, int& mine) {
  using K = typename KeyOf<R>::type;
  const float inf = topk_inf();
  const bool scored = A.bias != nullptr;  // selection values are scores plus bias
  K key[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    if (e >= A.experts) {
      key[i] = 0;
      continue;
    }
    R v = (R)x[i];
    if (scored) {
      const float b = A.bias[e];
      const bool masked = x[i] == -inf || !(b > -inf);
      v = masked ? (R)-inf : score_of<R>(x[i], norm, A.sigmoid) + (R)b;
    }
    key[i] = key_of(v);
  }

  bool open = false;
  // Bound of float32's error in a selection value below: the score's (a few
  // ulp of the largest score, plus the softmax sum's, 2^-24 for each of the
  // NV + 5 additions) and the rounding of the sum with the bias, 2^-24 of it.
  float eps = 0.f;
  if (sizeof(R) == 4 && (scored || A.group_top == 2))
    eps = A.sigmoid ? 0x1p-20f : 0x1p-18f / fmaxf((float)norm.total, 1.f);

  if (A.groups > 1) {
    // L lanes per group, each over a strided part of it, from the values in
    // shared memory; then the group's best two by shuffles.
    extern __shared__ __align__(16) unsigned char topk_smem[];
    R* row = reinterpret_cast<R*>(topk_smem) + (size_t)(threadIdx.x >> 5) * A.smem_row;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e = expert_at<VEC>(i, lane);
      if (e < A.experts) {
        R v = value_of(key[i]);
        if (A.group_top == 2 && !scored && x[i] != -inf) v = score_of<R>(x[i], norm, A.sigmoid);
        row[e + e / A.group_size] = v;  // one value of padding per group spreads them over the banks
      }
    }
    __syncwarp();
    const int L = A.lanes_per_group;
    const int g = lane / L;
    R b1 = (R)-inf, b2 = (R)-inf;
    if (g < A.groups)
      for (int j = lane % L; j < A.group_size; j += L) {
        const R v = row[g * (A.group_size + 1) + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
    for (int d = 1; d < L; d <<= 1) {
      const R o1 = __shfl_xor_sync(kFull, b1, d), o2 = __shfl_xor_sync(kFull, b2, d);
      const R lo = b1 < o1 ? b1 : o1;
      b1 = b1 < o1 ? o1 : b1;
      b2 = b2 < o2 ? o2 : b2;
      b2 = b2 < lo ? lo : b2;
    }
    const R val = b1 + (A.group_top == 2 && b2 > (R)-inf ? b2 : R(0));
    int ahead = 0;
    for (int h = 0; h < A.groups; h++) {
      const R o = __shfl_sync(kFull, val, h * L);
      ahead += (o > val || (o == val && h < g)) ? 1 : 0;
    }
    const bool in = g < A.groups && ahead < A.topk_groups;
    const unsigned chosen = __ballot_sync(kFull, in);
    if (eps > 0.f && A.topk_groups < A.groups) {
      // the last open group against the first closed one; each value is a sum
      // of up to two, each within eps and 2^-22 of its size
      const uint32_t ki = key_of((float)val);
      const float least = value_of(~warp_max(in ? ~ki : 0u));
      const float most = value_of(warp_max(in || g >= A.groups ? 0x007fffffu : ki));
      open = most > -inf && least - most <= 4.f * (eps + 0x1p-22f * fmaxf(fabsf(least), fabsf(most)));
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
      const int e = expert_at<VEC>(i, lane);
      if (e < A.experts && !((chosen >> ((e / A.group_size) * L)) & 1u)) key[i] = 0;
    }
  }

  K last = 0;
  for (int j = 0; j < A.topk; j++) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < NV; i++) best = key[i] > best ? key[i] : best;
    last = warp_max(best);
    uint32_t e = 0xffffffffu;
    if (best == last) {
#pragma unroll
      for (int i = NV - 1; i >= 0; i--)
        if (key[i] == last) e = (uint32_t)expert_at<VEC>(i, lane);
    }
    e = __reduce_min_sync(kFull, e);
    if (lane == j) mine = (int)e;
#pragma unroll
    for (int i = 0; i < NV; i++)
      if ((uint32_t)expert_at<VEC>(i, lane) == e) key[i] = 0;
  }
  if (sizeof(R) == 4 && scored) {
    // Neighbours of the selection (and the best value left out) closer than
    // their errors, unless logit and bias are equal: those are true ties.
    const bool have = lane < A.topk;
    const float xm = have ? logit_at<BF16>(logits, mine) : 0.f, bm = have ? A.bias[mine] : 0.f;
    const bool masked = !(xm > -inf) || !(bm > -inf);
    const float vm = !have || masked ? -inf : (float)(score_of<R>(xm, norm, A.sigmoid) + (R)bm);
    const float vn = __shfl_down_sync(kFull, vm, 1), xn = __shfl_down_sync(kFull, xm, 1),
                bn = __shfl_down_sync(kFull, bm, 1);
    const float top = __shfl_sync(kFull, vm, 0);
    const float end = value_of((uint32_t)last);
    const float xe = __shfl_sync(kFull, xm, A.topk - 1), be = __shfl_sync(kFull, bm, A.topk - 1);
    const float gap = 2.f * (eps + 0x1p-22f * fmaxf(fabsf(top), end > -inf ? fabsf(end) : 0.f));
    bool near = lane + 1 < A.topk && vm - vn <= gap && !(xm == xn && bm == bn);
    if (end > -inf) {
      uint32_t rest = 0;
#pragma unroll
      for (int i = 0; i < NV; i++)
        if (key[i] > rest && !(x[i] == xe && A.bias[expert_at<VEC>(i, lane)] == be)) rest = (uint32_t)key[i];
      rest = warp_max(rest);
      near = near || (rest > 0x007fffffu && end - value_of(rest) <= gap);
    }
    open = __any_sync(kFull, near) || open;
  }
  return open;
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

template <int NV, int VEC, bool BF16>
__device__ __noinline__ int select_row_f64(const TopkArgs& A, const char* logits, int lane, float most) {
  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; i++) {
    const int e = expert_at<VEC>(i, lane);
    const float v = e < A.experts ? logit_at<BF16>(logits, e) : -topk_inf();
    x[i] = v != v ? -topk_inf() : v;
  }
  int mine = 0;
  select_row<double, NV, VEC, BF16>(A, logits, x, lane, norm_of<double, NV>(x, most, !A.sigmoid), mine);
  return mine;
}

template <int NV, int VEC, bool BF16>
__global__ void __launch_bounds__(kTopkWarps * 32) k_topk(const __grid_constant__ TopkArgs A) {
  griddep_wait();
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
      if (BF16) {
        const uint4 v = ld_u4(logits + (size_t)e0 * 2);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < VEC; j++)
          x[c * VEC + j] = __uint_as_float((j & 1) ? (w[(j / 2) & 3] & 0xffff0000u) : (w[(j / 2) & 3] << 16));
      } else {
        const uint4 v = ld_u4(logits + (size_t)e0 * 4);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < VEC; j++) x[c * VEC + j] = __uint_as_float(w[j & 3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; j++) x[c * VEC + j] = e0 + j < A.experts ? logit_at<BF16>(logits, e0 + j) : -inf;
    }
  }
  uint32_t hi = 0;
#pragma unroll
  for (int i = 0; i < NV; i++) {
    if (x[i] != x[i]) x[i] = -inf;  // NaN counts as masked
    const uint32_t k = key_of(x[i]);
    hi = k > hi ? k : hi;
  }
  // softmax needs the row's maximum, and its sum where scores themselves count
  const bool scores = A.bias != nullptr || (A.groups > 1 && A.group_top == 2);
  const bool sum = !A.sigmoid && (scores || !A.renorm);
  const float most = sum ? value_of(warp_max(hi)) : 0.f;
  const Norm<float> norm = norm_of<float, NV>(x, most, sum);
  int mine = 0;
  if (select_row<float, NV, VEC, BF16>(A, logits, x, lane, norm, mine))
    mine = select_row_f64<NV, VEC, BF16>(A, logits, lane, most);

  // weights: lane j has expert j
  const bool have = lane < A.topk;
  float xm = have ? logit_at<BF16>(logits, mine) : -inf;
  if (have && A.bias && !(A.bias[mine] > -inf)) xm = -inf;
  if (!(xm > -inf)) xm = -inf;
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
