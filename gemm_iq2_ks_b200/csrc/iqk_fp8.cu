// 8-bit floating point (e4m3) with block scales: quantisation of activations,
// the product of two quantised operands, and the gate/up step of a dense
// expert (two products, SwiGLU, quantisation of the result).
//
// An activation row has one float32 scale per 128 columns, a weight matrix one
// per 128 x 128 block, so a product is
//   y[t][o] = sum_b xs[t][b] ws[o / 128][b] sum_{k in block b} xq[t][k] wq[o][k].
// The inner sums run on the tensor cores with float32 accumulators; the scales
// are applied to each 128-column block's sum in float32 on the way into the
// register accumulators.
#include <algorithm>
#include <atomic>

#include "iqk_device.cuh"
#include "iqk_internal.h"
#include "iqk_tc.cuh"

namespace iqk {

namespace {

__device__ int32_t g_fp8_status;  // nonzero once a bounded wait of a product expired

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 0x1p-100f;  // a group's largest magnitude counts as at least this

// Two e4m3 codes, nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// ------------------------------------------------------------- quantisation
//
// q = e4m3(448 x / m) with m the group's largest magnitude, exactly: the
// quotient of two bfloat16 numbers times 448 = 7 * 64 is either a rounding
// border of e4m3 (a number of at most 5 significant bits) or at least 2^-13
// of it away, because the difference 7 X 2^a - M B 2^b of integers with
// X, M < 2^8 and B < 2^5 is not zero and one of a, b is. x times the hardware's
// reciprocal is within 2^-22 of the quotient; rounding that to 18 significant
// bits (a step of at most 2^-17) returns a border exactly and keeps every
// other quotient on its side. This costs two integer operations instead of a
// division for each element: the kernel is bound by instructions (with IEEE
// divisions for the two scales and 8 elements a lane it issued 18 for each
// element and took 23.5 us for 8192 x 4096).
__device__ __forceinline__ float snap18(float t) {
  return __uint_as_float((__float_as_uint(t) + 0x20u) & ~0x3fu);
}
// 448 / m within 2^-22, for m from 2^-100 to the largest bfloat16 number; the
// scaling by 2^-8 keeps the reciprocal a normal number.
__device__ __forceinline__ float quick_inverse(float m) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(m * 0x1p-8f));
  return r * 1.75f;
}
// m / 448 rounded to nearest for a bfloat16 m: product with the rounded
// reciprocal and one correction by the fused remainder (Markstein 1990; exact
// for all 128 mantissas).
__device__ __forceinline__ float over_448(float m) {
  constexpr float r = 1.0f / 448.0f;
  const float q = m * r;
  return fmaf(fmaf(-448.0f, q, m), r, q);
}

constexpr int kQuantThreads = 256;
constexpr int kQuantLanes = 8;   // of a group of 128 columns, 16 columns (two 16-byte loads) each
constexpr int kQuantBlocks = 8;  // resident on an SM: 17.2 us for 8192 x 4096, 6 of them 17.4, two groups a lane 17.4

// A lane's next piece is on its way while the present one is converted.
__global__ void __launch_bounds__(kQuantThreads, kQuantBlocks)
    k_fp8_quantize(const uint16_t* x, int64_t stride, int cols, int nkb, FastDiv by_nkb, int items, uint8_t* q, float* s) {
  griddep_wait();
  griddep_launch();
  const int sub = threadIdx.x % kQuantLanes;
  const int per = gridDim.x * (kQuantThreads / kQuantLanes);
  struct Piece {
    uint4 v[2];
    int row, col;  // col past the end: nothing there
  };
  auto load = [&](Piece& g, int it) {
    g.row = (int)by_nkb.div((uint32_t)it);
    g.col = it < items ? (it - g.row * nkb) * kFp8Block + sub * 16 : cols;
    const uint4* p = reinterpret_cast<const uint4*>(x + g.row * stride + g.col);
#pragma unroll
    for (int j = 0; j < 2; j++) {
      g.v[j] = make_uint4(0, 0, 0, 0);
      if (g.col < cols) g.v[j] = p[j];
    }
  };
  int it = blockIdx.x * (kQuantThreads / kQuantLanes) + threadIdx.x / kQuantLanes;
  Piece cur, next;
  load(cur, it);
  for (; __any_sync(0xffffffffu, it < items); it += per) {
    load(next, it + per);
    uint32_t m2 = 0, o[4];
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const uint4 v = cur.v[j];
      m2 = __vmaxu2(__vmaxu2(m2, v.x & 0x7fff7fffu), v.y & 0x7fff7fffu);
      m2 = __vmaxu2(__vmaxu2(m2, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu);
    }
#pragma unroll
    for (int d = kQuantLanes / 2; d; d >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, d));
    const uint32_t mb = max(m2 & 0xffff0000u, m2 << 16);
    const bool fine = mb < 0x7f800000u;
    const float most = fmaxf(__uint_as_float(mb), kAmaxMin);
    const float inv = quick_inverse(most);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const uint32_t a = j & 1 ? cur.v[j / 2].z : cur.v[j / 2].x;
      const uint32_t b = j & 1 ? cur.v[j / 2].w : cur.v[j / 2].y;
      o[j] = e4m3x4(snap18(__uint_as_float(a << 16) * inv), snap18(__uint_as_float(a & 0xffff0000u) * inv),
                    snap18(__uint_as_float(b << 16) * inv), snap18(__uint_as_float(b & 0xffff0000u) * inv));
      o[j] = fine ? o[j] : 0u;
    }
    if (cur.col < cols) {
      *reinterpret_cast<uint4*>(q + (int64_t)cur.row * cols + cur.col) = make_uint4(o[0], o[1], o[2], o[3]);
      if (sub == 0) s[it] = fine ? over_448(most) : __int_as_float(0x7fffffff);
    }
    cur = next;
  }
}

// ------------------------------------------------------------------ products

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The two scales of a block's sum as factors, of which `big` is applied first
// and `small` in the multiply-add: 1 and their product where that is a normal
// number. Where it would overflow or lose bits (the sum times it may
// well be an ordinary number) the larger scale and the smaller one: block sums
// are 0 or between 2^-18 and 2^25, so no product on the way is out of range
// unless the result is.
struct Scale {
  float big, small;
};
__device__ __forceinline__ bool not_normal(float p) { return (((__float_as_uint(p) >> 23) + 1) & 255u) <= 1u; }
__device__ __forceinline__ Scale scale_of(float a, float b) {
  const float p = a * b;
  const bool far = not_normal(p) && a != 0.f && b != 0.f && fabsf(a) <= 3.402823466e38f && fabsf(b) <= 3.402823466e38f;
  const bool first = fabsf(a) >= fabsf(b);
  return {far ? (first ? a : b) : 1.f, far ? (first ? b : a) : p};
}

// Output element of the plain product.
__device__ __forceinline__ void put_y(const Fp8Args& A, int64_t i, float v) {
  if (A.f32) {
    if (A.add) v += static_cast<const float*>(A.add)[i];
    static_cast<float*>(A.y)[i] = v;
  } else {
    if (A.add) v += bf16_bits_to_f32(static_cast<const uint16_t*>(A.add)[i]);
    static_cast<uint16_t*>(A.y)[i] = f32_to_bf16_bits(v);
  }
}

__device__ __forceinline__ float magnitude(float h) {  // infinity for what is not finite
  const float m = fabsf(h);
  return m <= 3.402823466e38f ? m : __int_as_float(0x7f800000);
}

// ----------------------------------------------------------- many tokens
//
// tcgen05 tiles of 128 tokens x BN weight rows (gate_up: 128 gate and 128 up
// rows side by side). One 128-column block is one pipeline step: TMA brings
// both operands' 128-byte rows (128-byte swizzle), four MMAs leave the block's
// sums in one of the tensor-memory buffers, and 16 warps add them, times the
// two scales, to float32 accumulators in registers (thread = token row; a
// quarter of the columns for each four warps). CTAs are persistent over tiles:
// the copies and MMAs of the next tile run while this one is stored. With few
// tiles the CTAs of a cluster split the blocks of one tile and add their
// accumulators over distributed shared memory, in rank order. With many, two
// CTAs form a pair (PAIR, cta_group::2) on 256 tokens x 256 rows: each holds
// its tokens and half of the weight rows, which halves what an MMA reads of
// shared memory for its weights (128 x 256 x 32 alone took 196 cycles, of 128
// that the tensor cores need).
//
// What bounds it is the hand-over of the accumulators: a step's sums (128 rows x
// 256 columns, 128 KB for each CTA of a pair) have to leave tensor memory before
// the MMAs of the second next step; a step takes 940 cycles, its MMAs 512. What
// counted there, measured at 8192 x 4096 x 4096: the token scales go through
// shared memory (each row of a warp's direct load is a line of its own: +12%),
// on the barrier that the step waits for anyway (a barrier of their own: +20%),
// the larger factors of far scales are read beside them (a flag read ahead of
// the loads instead: +8%), arrivals and waits have CTA scope (what they order is
// tensor memory, by its own fences; cluster scope took twice the time), and no
// register of the loop is spilled (+10 to 20% for a few bytes). 125 us on
// operands of small codes (2.20 PFLOP/s); quantised normal data takes 132 to
// 152 us at the same instructions, the longer it runs, by the card's power limit.
constexpr int kBM = 128;
constexpr int kEpiWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kScaleWarp = 18;  // and 19
constexpr int kGemmThreads = 20 * 32;
// Registers: 640 threads are launched with 96 each; the accumulating warps take
// 112, the last warpgroup keeps 32 (4 x 112 + 32 = 5 x 96).
constexpr int kEpiRegs = 112, kLastRegs = 32;
constexpr int kGemmStageBytes(int BN, bool pair) { return (kBM + (pair ? BN / 2 : BN)) * kFp8Block; }
constexpr int kGemmRing(int BN, bool pair) { return (BN == 256 && !pair ? 4 : 5) * kGemmStageBytes(BN, pair); }
constexpr int kPitch(int BN) { return BN + 4; }  // floats between rows of the shared accumulators
constexpr int kStageOut = 2048;                  // bytes of one warp's store staging: 32 rows x 16 floats
constexpr int kStaging(bool gu) { return gu ? 4 * kBM * 4 : kEpiWarps * kStageOut; }
// With the scales of a step beside each accumulator: [2 weight blocks][128 rows]
// products of token and block scale (or the smaller of the two, and the larger
// one in a second table, see scale_of), written by two warps of their own.
constexpr size_t kGemmSmem(int BN, bool gu, bool pair) {
  return kGemmRing(BN, pair) + kStaging(gu) + 2 * (512 / BN * 2 * kBM * 4) + 256 + 1024;
}
static_assert(kBM * kPitch(256) * 4 <= kGemmRing(256, false) && kBM * kPitch(128) * 4 <= kGemmRing(128, false),
              "accumulators");

// Bounded wait of a whole warp: gives up, every lane alike, once `limit_ns` of
// the GPU's global timer have passed, or soon after another warp of the CTA did.
__device__ __forceinline__ bool gemm_wait(uint64_t* bar, uint32_t par, volatile uint32_t* abort_flag, uint64_t limit_ns) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
    const bool late = globaltimer_ns() - t0 >= limit_ns;
    if (__any_sync(0xffffffffu, late || *abort_flag)) {
      if (late) {
        *abort_flag = 1;
        atomicOr(&g_fp8_status, 2);
      }
      return false;
    }
  }
}

template <bool PAIR = false>
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two CTAs of a cluster as one (cta_group::2): tensor memory, the copy whose
// bytes count on the first CTA's barrier, the commit that arrives in both, the
// arrival in the first.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* holder_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t base, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of a converged warp: the copies and MMAs are issued under it, from
// code that the whole warp runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// The wait names the loaded registers, so that nothing reads them ahead of it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The warp's lanes of N columns times big(column), in tensor memory: for the few
// steps of few-token products whose scales are not applied as one factor
// (scale_of). It stands ahead of the ordinary path, whose registers stay as
// they are.
template <int N, typename F>
__device__ __forceinline__ void scale_tmem(uint32_t taddr, F big) {
#pragma unroll 1
  for (int c0 = 0; c0 < N; c0 += 8) {
    float v[8];
    tmem_ld8(taddr + c0, v);
#pragma unroll
    for (int c = 0; c < 8; c++) v[c] *= big(c0 + c);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr + c0),
                 "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  }
  tmem_wait_st();
}

// Two float32 fused multiply-adds in one instruction: acc += (lo, hi) * (s, s).
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(s));
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// The same for 32 columns straight from tensor memory, as one block: the loaded
// registers stay in it, paired where they are (the separate forms copy them
// first).
// `sc`: shared-memory address of the row's factor `small`, `big` BIG bytes
// behind it (scale_of); both are on their way while the sums are.
#define IQK_FMA2(lo, hi, a) "mov.b64 p, {t" lo ", t" hi "};\n\tfma.rn.f32x2 %" a ", p, s, %" a ";\n\t"
#define IQK_MUL(i) "mul.rn.f32 t" i ", t" i ", g;\n\t"
template <int BIG>
__device__ __forceinline__ void ld_fma32(uint32_t taddr, uint64_t* a, uint32_t sc) {
  asm volatile(
      "{\n\t.reg .b32 t<32>;\n\t.reg .b64 p, s;\n\t.reg .f32 f, g;\n\t.reg .pred q;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, "
      "t12, t13, t14, t15, t16, t17, t18, t19, t20, t21, t22, t23, "
      "t24, t25, t26, t27, t28, t29, t30, t31}, [%16];\n\t"
      "ld.shared.f32 f, [%17];\n\tld.shared.f32 g, [%17+%18];\n\t"
      "mov.b64 s, {f, f};\n\t"
      "setp.neu.f32 q, g, 0f3f800000;\n\t"
      "vote.sync.any.pred q, q, 0xffffffff;\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "@!q bra.uni ONE_%=;\n\t"
      IQK_MUL("0") IQK_MUL("1") IQK_MUL("2") IQK_MUL("3")
      IQK_MUL("4") IQK_MUL("5") IQK_MUL("6") IQK_MUL("7")
      IQK_MUL("8") IQK_MUL("9") IQK_MUL("10") IQK_MUL("11")
      IQK_MUL("12") IQK_MUL("13") IQK_MUL("14") IQK_MUL("15")
      IQK_MUL("16") IQK_MUL("17") IQK_MUL("18") IQK_MUL("19")
      IQK_MUL("20") IQK_MUL("21") IQK_MUL("22") IQK_MUL("23")
      IQK_MUL("24") IQK_MUL("25") IQK_MUL("26") IQK_MUL("27")
      IQK_MUL("28") IQK_MUL("29") IQK_MUL("30") IQK_MUL("31")
      "ONE_%=:\n\t"
      IQK_FMA2("0", "1", "0")
      IQK_FMA2("2", "3", "1")
      IQK_FMA2("4", "5", "2")
      IQK_FMA2("6", "7", "3")
      IQK_FMA2("8", "9", "4")
      IQK_FMA2("10", "11", "5")
      IQK_FMA2("12", "13", "6")
      IQK_FMA2("14", "15", "7")
      IQK_FMA2("16", "17", "8")
      IQK_FMA2("18", "19", "9")
      IQK_FMA2("20", "21", "10")
      IQK_FMA2("22", "23", "11")
      IQK_FMA2("24", "25", "12")
      IQK_FMA2("26", "27", "13")
      IQK_FMA2("28", "29", "14")
      IQK_FMA2("30", "31", "15")
      "}"
      : "+l"(a[0]), "+l"(a[1]), "+l"(a[2]), "+l"(a[3]), "+l"(a[4]), "+l"(a[5]), "+l"(a[6]), "+l"(a[7]),
        "+l"(a[8]), "+l"(a[9]), "+l"(a[10]), "+l"(a[11]), "+l"(a[12]), "+l"(a[13]), "+l"(a[14]), "+l"(a[15])
      : "r"(taddr), "r"(sc), "n"(BIG));
}
#undef IQK_MUL
#undef IQK_FMA2

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (format code 0), float32
// accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t m, uint32_t n) {
  return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Four neighbouring outputs of one row; A.vec: rows and pointers allow vector access.
__device__ __forceinline__ void put_y4(const Fp8Args& A, int64_t t, int n, float4 v) {
  const int64_t i = t * A.rows + n;
  if (!A.vec) {
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 4; c++)
      if (n + c < A.rows) put_y(A, i + c, w[c]);
    return;
  }
  if (n >= A.rows) return;
  if (A.f32) {
    if (A.add) {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(A.add) + i);
      v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
    }
    *reinterpret_cast<float4*>(static_cast<float*>(A.y) + i) = v;
  } else {
    if (A.add) {
      const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(A.add) + i);
      v.x += __uint_as_float(a.x << 16);
      v.y += __uint_as_float(a.x & 0xffff0000u);
      v.z += __uint_as_float(a.y << 16);
      v.w += __uint_as_float(a.y & 0xffff0000u);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + i) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

constexpr int kMaxSplit = 8;  // CTAs of a cluster

// One warp ends one token's row of V * 128 columns: the sum over the cluster's
// CTAs of the accumulators at `src` in each one's shared memory, in rank order,
// and what becomes of it. Gate_up: 128 gate columns, then their up columns.
// WIDE: all loads on their way before the first is used, where there are
// registers for it (0.7 us less for gate_up of 1 token).
template <int V, bool GU, bool WIDE>
__device__ __forceinline__ void finish_row(const Fp8Args& A, const float* src, int split, int64_t t, int n0, int lane) {
  float4 v[V];
#pragma unroll
  for (int h = 0; h < V; h++) {
    v[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (split == 1) {
      v[h] = *reinterpret_cast<const float4*>(src + 128 * h + 4 * lane);
    } else if (!WIDE) {
      for (int k = 0; k < split; k++) {
        const float4 o = ld_peer4(peer_smem(src + 128 * h + 4 * lane, k));
        v[h].x += o.x;
        v[h].y += o.y;
        v[h].z += o.z;
        v[h].w += o.w;
      }
    }
  }
  if (WIDE && split > 1) {
    float4 o[kMaxSplit][V];
#pragma unroll
    for (int k = 0; k < kMaxSplit; k++)
#pragma unroll
      for (int h = 0; h < V; h++)
        if (k < split) o[k][h] = ld_peer4(peer_smem(src + 128 * h + 4 * lane, k));
#pragma unroll
    for (int k = 0; k < kMaxSplit; k++)
#pragma unroll
      for (int h = 0; h < V; h++)
        if (k < split) {
          v[h].x += o[k][h].x;
          v[h].y += o[k][h].y;
          v[h].z += o[k][h].z;
          v[h].w += o[k][h].w;
        }
  }
  const int n = n0 + 4 * lane;
  if (GU) {
    const float4 gv = v[0], uv = v[V - 1];
    const float h0 = silu_f32(gv.x) * uv.x, h1 = silu_f32(gv.y) * uv.y, h2 = silu_f32(gv.z) * uv.z,
                h3 = silu_f32(gv.w) * uv.w;
    float most = n < A.rows ? fmaxf(fmaxf(magnitude(h0), magnitude(h1)), fmaxf(magnitude(h2), magnitude(h3))) : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    const bool fine = most <= 3.402823466e38f;
    most = fmaxf(most, kAmaxMin);
    const float inv = fine ? kE4m3Max / most : 0.f;
    const uint32_t o = fine ? e4m3x4(h0 * inv, h1 * inv, h2 * inv, h3 * inv) : 0u;
    if (n < A.rows) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(A.y) + t * A.rows + n) = o;
    if (lane == 0)
      A.hs[t * ((A.rows + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block] =
          fine ? most / kE4m3Max : __int_as_float(0x7fffffff);
  } else {
#pragma unroll
    for (int h = 0; h < V; h++) put_y4(A, t, n + 128 * h, v[h]);
  }
}

// After a wait of a pair expired, when both CTAs have stopped: lets the products
// and the copies in flight end. The copies of both CTAs count on the first one's
// barriers, each step's as 2 x SB bytes that the first CTA expects; where the
// CTAs stopped at different steps (by at most the ring's depth), it accounts
// for what is missing.
template <int ST, int SB>
__device__ __forceinline__ void drain_pair(uint64_t* full, uint64_t* drain, int n0, int n1, int half, bool copies,
                                           bool products) {
  if (products) {
    if (half == 0 && elect_one()) tc_commit_pair(drain);
    __syncwarp();
    mbar_wait_ns(drain, 0, kDrainWaitNs);
  }
  if (copies && half == 0) {
    const int most = max(n0, n1);
    if (elect_one())
      for (int j = min(n0, n1); j < most; j++) {
        if (n0 < n1)
          mbar_arrive_expect_tx(&full[j % ST], SB);  // the second CTA's copies alone
        else
          mbar_complete_tx(&full[j % ST], SB);  // copies that the second CTA did not begin
      }
    __syncwarp();
    for (int j = most < ST ? 0 : most - ST; j < most; j++) mbar_wait_ns(&full[j % ST], (j / ST) & 1, kDrainWaitNs);
  }
}

template <int BN, bool GU, bool PAIR>
__global__ void __launch_bounds__(kGemmThreads, 1)
    k_fp8_gemm(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap m0,
               const __grid_constant__ CUtensorMap m1, const __grid_constant__ Fp8Args A, int tiles_m, int tiles,
               int split) {
  constexpr int SB = kGemmStageBytes(BN, PAIR), ST = kGemmRing(BN, PAIR) / SB, NC = BN / 4;
  constexpr int NBUF = 512 / BN;  // accumulators in tensor memory
  constexpr int NB = GU ? 128 : BN;  // output columns of a tile
  static_assert(BN == (GU || PAIR ? 256 : 128), "the forms that launch_fp8_product takes");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* staging = smem + kGemmRing(BN, PAIR);
  float* scales = reinterpret_cast<float*>(staging + kStaging(GU));
  constexpr int kBigs = NBUF * 2 * kBM;  // behind the table of the smaller factors: that of the larger ones
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + 2 * kBigs);
  uint64_t* empty = full + ST;
  uint64_t* tfull = empty + ST;
  uint64_t* tfree = tfull + NBUF;
  uint64_t* sfree = tfree + NBUF;
  uint64_t* drain = sfree + NBUF;
  uint64_t* never = drain + 1;  // nothing arrives on it (testing hook)
  uint32_t* holder = reinterpret_cast<uint32_t*>(never + 1);
  volatile uint32_t* abort_flag = holder + 1;
  volatile uint32_t* copied = holder + 2;  // PAIR: steps that each CTA has copied; the top bit: it gave up
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // PAIR: `split` is 1 and the cluster's two CTAs take the halves of a tile's 256 tokens.
  const int rank = split > 1 ? (int)cluster_rank() : 0, half = PAIR ? (int)cluster_rank() : 0;
  const int group = PAIR ? 2 : split;
  const int first = blockIdx.x / group, step = gridDim.x / group;
  const int kb_lo = (int)((int64_t)A.nkb * rank / split), kb_hi = (int)((int64_t)A.nkb * (rank + 1) / split);
  const int steps = kb_hi - kb_lo;

  if (warp == 0) {  // the barriers lie one after the other, a lane for each
    constexpr int T0 = 2 * ST, T1 = T0 + NBUF, T2 = T1 + NBUF, T3 = T2 + NBUF;  // from T3: drain, never
    static_assert(T3 + 1 < 32 && (T3 + 2) * 8 + 16 <= 256, "barriers");
    if (lane <= T3 + 1)
      mbar_init(&full[lane], lane < T0    ? 1
                             : lane < T1  ? 3  // tfull: the commit and the two scale warps
                             : lane < T2  ? (PAIR ? 2 * kEpiWarps : kEpiWarps)
                             : lane < T3  ? kEpiWarps
                                          : 1);
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tensormap(&mx);
    prefetch_tensormap(&m0);
    prefetch_tensormap(&m1);
  }
  if (warp == kMmaWarp) {
    if (PAIR)
      tmem_alloc_pair(holder, 512);
    else
      tmem_alloc(holder, 512);
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) {  // both CTAs' barriers and tensor memory are ready
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_after();
  const uint32_t tmem = *holder;
  griddep_wait();
  griddep_launch();

  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLastRegs));
    if (warp == kTmaWarp) {
      const bool leader = elect_one();
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int t0 = (tile % tiles_m * (PAIR ? 2 : 1) + half) * kBM, n0 = (tile / tiles_m) * NB;
        for (int i = 0; i < steps; i++, it++) {
          const int s = it % ST, k = (kb_lo + i) * kFp8Block;
          if (!(ok = gemm_wait(&empty[s], ((it / ST) & 1) ^ 1, abort_flag, A.wait_ns))) break;
          if (leader) {
            uint8_t* a = smem + s * SB;
            uint8_t* w = a + kBM * kFp8Block;
            if (PAIR) {  // each CTA: its tokens and half of the weight rows (gate_up: gate or up)
              if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * SB);
              const uint32_t bar = peer_smem(&full[s], 0);
              tma_load_2d_pair(a, &mx, k, t0, bar);
              tma_load_2d_pair(w, GU && half ? &m1 : &m0, k, GU ? n0 : n0 + 128 * half, bar);
            } else {
              mbar_arrive_expect_tx(&full[s], SB);
              tma_load_2d(a, &mx, k, t0, &full[s]);
              tma_load_2d(w, &m0, k, n0, &full[s]);
              if (GU) tma_load_2d(w + 128 * kFp8Block, &m1, k, n0, &full[s]);
            }
          }
          __syncwarp();
        }
      }
      // The last stages' commits arrive here, too: nothing may exit before they have.
      for (int j = it < ST ? 0 : it - ST; ok && j < it; j++)
        ok = gemm_wait(&empty[j % ST], (j / ST) & 1, abort_flag, A.wait_ns);
      if (!ok && !PAIR)  // a wait expired: let the copies in flight land
        for (int j = it < ST ? 0 : it - ST; j < it; j++) mbar_wait_ns(&full[j % ST], (j / ST) & 1, kDrainWaitNs);
      if (PAIR && leader) {  // both CTAs learn of it; see drain_pair below
        const uint32_t v = (uint32_t)it | (ok ? 0u : 0x80000000u);
        st_peer(peer_smem(holder + 2 + half, 0), v);
        st_peer(peer_smem(holder + 2 + half, 1), v);
      }
    }
    if (warp == kMmaWarp && half == 0) {
      const bool leader = elect_one();
      // descriptors differ in the address field (bytes / 16) only
      const uint64_t d0 = sdesc_kmajor_sw128(smem_u32(smem));
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        for (int i = 0; i < steps; i++, it++) {
          const int s = it % ST, b = it % NBUF;
          if (!(ok = gemm_wait(&full[s], (it / ST) & 1, abort_flag, A.wait_ns) &&
                     gemm_wait(&tfree[b], ((it / NBUF) & 1) ^ 1, abort_flag, A.wait_ns)))
            break;
          tc_fence_after();
          if (leader) {
            const uint64_t da = d0 + (uint32_t)(s * (SB / 16)), dw = da + kBM * kFp8Block / 16;
#pragma unroll
            for (int j = 0; j < 4; j++)
              mma_ss_e4m3<PAIR>(tmem + b * BN, da + 2u * j, dw + 2u * j, idesc_e4m3(PAIR ? 256 : 128, BN), j != 0);
            if (PAIR) {
              tc_commit_pair(&tfull[b]);
              tc_commit_pair(&empty[s]);
            } else {
              tc_commit(&tfull[b]);
              tc_commit(&empty[s]);
            }
          }
          __syncwarp();
        }
      }
      if (!ok && !PAIR) {  // a wait expired: let the products in flight end before their tensor memory is given back
        if (leader) tc_commit(drain);
        mbar_wait_ns(drain, 0, kDrainWaitNs);
      }
    }
    if (warp >= kScaleWarp) {
      // rows 64 w + lane and 32 on, one step's scales fetched ahead
      const int r = 64 * (warp - kScaleWarp) + lane;
      uint32_t dirty = ~0u;  // accumulators whose table of larger factors is not all 1
      int it = 0;
      bool ok = true;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int t0 = (tile % tiles_m * (PAIR ? 2 : 1) + half) * kBM, n0 = (tile / tiles_m) * NB;
        const int last = (A.rows - 1) / kFp8Block;  // blocks past it: any, their columns are not stored
        uint32_t x0 = (uint32_t)min(t0 + r, A.T - 1) * A.nkb + kb_lo, x1 = (uint32_t)min(t0 + r + 32, A.T - 1) * A.nkb + kb_lo;
        const uint32_t w0 = (uint32_t)min(n0 / kFp8Block, last) * A.nkb + kb_lo;
        const uint32_t w1 = (uint32_t)min(n0 / kFp8Block + (GU ? 0 : 1), last) * A.nkb + kb_lo;
        float a0 = A.xs[x0], a1 = A.xs[x1];
        for (int i = 0; i < steps; i++, it++) {
          const float b0 = A.w0.s[w0 + i], b1 = (GU ? A.w1.s : A.w0.s)[w1 + i];
          if (i + 1 < steps) {
            x0++;
            x1++;
          }
          const float na0 = A.xs[x0], na1 = A.xs[x1];
          if (!(ok = gemm_wait(&(PAIR ? sfree : tfree)[it % NBUF], ((it / NBUF) & 1) ^ 1, abort_flag, A.wait_ns)))
            break;
          float* dst = scales + (it % NBUF) * 2 * kBM + r;
          bool far = false;
          auto each = [&](auto f) {
            f(0, a0, b0);
            f(32, a1, b0);
            if (BN == 256) {
              f(kBM, a0, b1);
              f(kBM + 32, a1, b1);
            }
          };
          each([&](int i, float a, float b) {
            dst[i] = a * b;
            far |= not_normal(a * b);
          });
          if (__any_sync(0xffffffffu, far) || (dirty >> (it % NBUF) & 1)) {
            far = false;
            each([&](int i, float a, float b) {
              const Scale f = scale_of(a, b);
              dst[i] = f.small;
              dst[kBigs + i] = f.big;
              far |= f.big != 1.f;
            });
            dirty = (dirty & ~(1u << it % NBUF)) | (uint32_t)(__any_sync(0xffffffffu, far) != 0) << it % NBUF;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&tfull[it % NBUF]);
          a0 = na0;
          a1 = na1;
        }
      }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (PAIR) {  // neither CTA's memory is in use any more
      cluster_arrive();
      cluster_wait();
      if ((copied[0] | copied[1]) >> 31) {
        drain_pair<ST, SB>(full, drain, copied[0] & 0x7fffffffu, copied[1] & 0x7fffffffu, half,
                           warp == kTmaWarp, warp == kMmaWarp);
        cluster_arrive();
        cluster_wait();
      }
      if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
      return;
    }
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    if (split > 1) {  // the two cluster barriers of the other warps
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
  {
    // Lanes 32 q .. 32 q + 31 of tensor memory; columns part * NC and on of the
    // block, for gate_up 32 gate columns and the same 32 up columns.
    const int q = warp & 3, part = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
    int it = 0;
    bool ok = true;  // after an expired wait the barriers are kept, the work is not
    if (A.expire && warp == 0) ok = gemm_wait(never, 0, abort_flag, A.wait_ns);  // testing hook: this wait runs out
    for (int tile = first; tile < tiles; tile += step) {
      const int t0 = (tile % tiles_m * (PAIR ? 2 : 1) + half) * kBM, n0 = (tile / tiles_m) * NB;
      const int t = t0 + 32 * q + lane;
      const bool rows_in = t0 + 32 * q < A.T;  // some row of this warp exists
      uint64_t acc[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; c++) acc[c] = 0;
      for (int i = 0; i < steps; i++, it++) {
        const int b = it % NBUF;
        if (!(ok = ok && gemm_wait(&tfull[b], (it / NBUF) & 1, abort_flag, A.wait_ns))) continue;
        tc_fence_after();
        const float* sc = scales + b * 2 * kBM + (BN == 256 && !GU && part >= 2 ? kBM : 0) + 32 * q + lane;
        if (rows_in) {
          const uint32_t col = lanes + b * BN + (GU ? part * 32 : part * NC);
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 32)
            ld_fma32<kBigs * 4>(col + (GU && c0 ? 128 : c0), acc + c0 / 2, smem_u32(sc) + (GU && c0 ? kBM * 4 : 0));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // the accumulator and its scales are free
          if (PAIR) {
            mbar_arrive_peer(peer_smem(&tfree[b], 0));
            mbar_arrive(&sfree[b]);
          } else {
            mbar_arrive(&tfree[b]);
          }
        }
      }
      if (split > 1) {
        // All MMAs have read their operands: the ring takes the accumulators.
        if (rows_in && ok) {
          float* dst = reinterpret_cast<float*>(smem) + (size_t)(32 * q + lane) * kPitch(BN);
#pragma unroll
          for (int c = 0; c < NC; c += 4)
            *reinterpret_cast<float4*>(dst + (GU ? part * 32 + (c < 32 ? c : 96 + c) : part * NC + c)) =
                make_float4(lo_of(acc[c / 2]), hi_of(acc[c / 2]), lo_of(acc[c / 2 + 1]), hi_of(acc[c / 2 + 1]));
        }
      } else if (GU) {
        // h in the thread; the row's largest magnitude over the four warps with its columns
        float h[32], most = 0.f;
        const int n = n0 + part * 32;
#pragma unroll
        for (int c = 0; c < 32; c++) {
          const float g = (c & 1) ? hi_of(acc[c / 2]) : lo_of(acc[c / 2]);
          const float u = (c & 1) ? hi_of(acc[NC / 4 + c / 2]) : lo_of(acc[NC / 4 + c / 2]);
          h[c] = silu_f32(g) * u;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 16)  // rows is a multiple of 16
          if (n + c < A.rows) {
#pragma unroll
            for (int j = 0; j < 16; j++) most = fmaxf(most, magnitude(h[c + j]));
          }
        float* smost = reinterpret_cast<float*>(staging);  // [4 parts][128 rows]
        smost[part * kBM + 32 * q + lane] = most;
        asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
#pragma unroll
        for (int k = 0; k < 4; k++) most = fmaxf(most, smost[k * kBM + 32 * q + lane]);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory");
        const bool fine = most <= 3.402823466e38f;
        most = fmaxf(most, kAmaxMin);
        const float inv = fine ? kE4m3Max / most : 0.f;
        if (t < A.T) {
#pragma unroll
          for (int c = 0; c < 32; c += 16)
            if (n + c < A.rows) {
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; j++)
                o[j] = fine ? e4m3x4(h[c + 4 * j] * inv, h[c + 4 * j + 1] * inv, h[c + 4 * j + 2] * inv,
                                     h[c + 4 * j + 3] * inv)
                            : 0u;
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(A.y) + (int64_t)t * A.rows + n + c) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          if (part == 0)
            A.hs[(int64_t)t * ((A.rows + kFp8Block - 1) / kFp8Block) + n0 / kFp8Block] =
                fine ? most / kE4m3Max : __int_as_float(0x7fffffff);
        }
      } else if (rows_in) {
        // Through the warp's staging, 16 columns at a time, to stores of whole
        // 32-byte sectors; 16-byte pieces are permuted against bank conflicts.
        float* st = reinterpret_cast<float*>(staging + warp * kStageOut);
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += 16) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const int c = (c0 + 4 * j) / 2;
            *reinterpret_cast<float4*>(st + lane * 16 + 4 * (j ^ ((lane >> 1) & 3))) =
                make_float4(lo_of(acc[c]), hi_of(acc[c]), lo_of(acc[c + 1]), hi_of(acc[c + 1]));
          }
          __syncwarp();
          // Not unrolled in full: this code runs once a tile, and fetching it costs
          // more than its loop (4099 x 2196 x 528: 20.1 to 18.9 us). Without vector
          // access a lane takes a column, so that a store instruction covers two
          // runs of 16 and not eight of every fourth element (rows 2197: 47.8 to 29.1 us).
          if (!A.vec) {
            const int c = lane & 15, n = n0 + part * NC + c0 + c;
#pragma unroll 4
            for (int r = lane >> 4; r < 32; r += 2) {
              const float v = st[r * 16 + 4 * ((c >> 2) ^ ((r >> 1) & 3)) + (c & 3)];
              const int64_t tr = t0 + 32 * q + r;
              if (tr < A.T && n < A.rows) put_y(A, tr * A.rows + n, v);
            }
            continue;
          }
#pragma unroll 1
          for (int i = 0; i < 4; i++) {
            const int r = 8 * i + (lane >> 2), j = lane & 3;
            const float4 v = *reinterpret_cast<const float4*>(st + r * 16 + 4 * (j ^ ((r >> 1) & 3)));
            const int64_t tr = t0 + 32 * q + r;
            if (tr < A.T) put_y4(A, tr, n0 + part * NC + c0 + 4 * j, v);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (PAIR) {
    cluster_arrive();
    cluster_wait();
    if ((copied[0] | copied[1]) >> 31) {  // the other warps drain
      cluster_arrive();
      cluster_wait();
    }
  }
  if (split == 1) return;

  cluster_arrive();
  cluster_wait();
  // One warp per row, rows dealt to the cluster's CTAs and their warps in turn.
  const int t0 = (first % tiles_m) * kBM, n0 = (first / tiles_m) * NB;
  const int nrow = min(kBM, A.T - t0);
  for (int r = rank + split * warp; r < nrow; r += split * kEpiWarps)
    finish_row<BN / 128, GU, false>(A, reinterpret_cast<const float*>(smem) + (size_t)r * kPitch(BN), split, t0 + r, n0, lane);
  cluster_arrive();  // the peers have read this CTA's accumulators
  cluster_wait();
}

// ---------------------------------------------------------------- few tokens
//
// The same with the operands' places changed: M = 128 weight rows (gate_up: two
// MMAs, of 128 gate and of 128 up rows), N = the tokens, padded to TN. A step
// then costs the tensor cores what its weights' bytes cost to read, where 128
// token rows would be mostly padding. Thread = weight row; the token scales,
// times the block's, come from a table that each warp writes for each step.
// A latency chain bounds it (start, first copies, a few steps, the exchange in
// the cluster): 4096 x 4096 takes 4.8 us for 1 token and 6.3 us for 32 (3.5 and
// 2.7 TB/s, operands in L2; 5.8 and 7.3 us over three sets of them), where a
// 64-token form took 8.2 us, no less than the tiles above, and a stream over
// the weights with mma.sync 5.1 us for 1 and 10.9 for 16.
constexpr int kSkinnyThreads = 6 * 32;
constexpr int kSkinnyMaxT = 32;
constexpr int kSkStage(bool gu, int TN) { return ((gu ? 256 : 128) + TN) * kFp8Block; }
constexpr int kSkStages(bool gu) { return gu ? 3 : 5; }
constexpr int kSkBufs = 4;  // accumulators in tensor memory: at most 256 columns for each of two CTAs
constexpr int kSkRing(bool gu, int TN) { return kSkStages(gu) * kSkStage(gu, TN); }
constexpr size_t kSkSmem(bool gu, int TN) { return kSkRing(gu, TN) + 2 * (4 * 2 * kSkinnyMaxT * 4) + 256 + 1024; }
static_assert(kSkRing(true, 32) >= 32 * 256 * 4 && kSkRing(false, 32) >= 32 * 128 * 4, "accumulators");
// Two CTAs fit on an SM by shared memory, registers and tensor memory; how many
// clusters do is asked of the runtime (pick_split: 16 tiles of gate_up get
// clusters of 6, 96 CTAs).
static_assert(kSkSmem(true, 32) <= 113 * 1024 && kSkSmem(false, 32) <= 113 * 1024, "two CTAs on an SM");

template <bool GU, int TN>
__global__ void __launch_bounds__(kSkinnyThreads, 2)
    k_fp8_skinny(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap m0,
                 const __grid_constant__ CUtensorMap m1, const __grid_constant__ Fp8Args A, int split) {
  constexpr int M = GU ? 2 : 1, ST = kSkStages(GU), SB = kSkStage(GU, TN), NBUF = kSkBufs;
  constexpr int COLS = NBUF * TN * M, LD = TN < 32 ? 16 : 32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* table = reinterpret_cast<float*>(smem + kSkRing(GU, TN));  // [4 warps][2][32]
  constexpr int kBigs = 4 * 2 * kSkinnyMaxT;  // a second one behind it, for the larger scales (scale_of)
  uint64_t* full = reinterpret_cast<uint64_t*>(table + 2 * kBigs);
  uint64_t* empty = full + ST;
  uint64_t* tfull = empty + ST;
  uint64_t* tfree = tfull + NBUF;
  uint64_t* drain = tfree + NBUF;
  uint64_t* never = drain + 1;  // nothing arrives on it (testing hook)
  uint32_t* holder = reinterpret_cast<uint32_t*>(never + 1);
  volatile uint32_t* abort_flag = holder + 1;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int n0 = (int)(blockIdx.x / split) * 128;
  const int kb_lo = (int)((int64_t)A.nkb * rank / split), kb_hi = (int)((int64_t)A.nkb * (rank + 1) / split);
  const int steps = kb_hi - kb_lo;

  if (warp == 0) {  // the barriers lie one after the other, a lane for each
    constexpr int T0 = 2 * ST + NBUF, T1 = T0 + NBUF;
    static_assert(T1 + 1 < 32 && (T1 + 2) * 8 + 8 <= 256, "barriers");
    if (lane <= T1 + 1) mbar_init(&full[lane], lane >= T0 && lane < T1 ? 4 : 1);  // tfree: four warps
    if (lane == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&mx);
    prefetch_tensormap(&m0);
    prefetch_tensormap(&m1);
  }
  if (warp == 5) tmem_alloc(holder, COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  griddep_wait();
  griddep_launch();

  if (warp == 4) {
    const bool leader = elect_one();
    int i = 0;
    bool ok = true;
    for (; i < steps; i++) {
      const int s = i % ST, k = (kb_lo + i) * kFp8Block;
      if (!(ok = gemm_wait(&empty[s], ((i / ST) & 1) ^ 1, abort_flag, A.wait_ns))) break;
      if (leader) {
        uint8_t* a = smem + s * SB;
        mbar_arrive_expect_tx(&full[s], SB);
        tma_load_2d(a, &m0, k, n0, &full[s]);
        if (GU) tma_load_2d(a + 128 * kFp8Block, &m1, k, n0, &full[s]);
        tma_load_2d(a + M * 128 * kFp8Block, &mx, k, 0, &full[s]);
      }
      __syncwarp();
    }
    // The last stages' commits arrive here, too: nothing may exit before they have.
    for (int j = i < ST ? 0 : i - ST; ok && j < i; j++)
      ok = gemm_wait(&empty[j % ST], (j / ST) & 1, abort_flag, A.wait_ns);
    if (!ok)  // a wait expired: let the copies in flight land
      for (int j = i < ST ? 0 : i - ST; j < i; j++) mbar_wait_ns(&full[j % ST], (j / ST) & 1, kDrainWaitNs);
  } else if (warp == 5) {
    const bool leader = elect_one();
    const uint64_t d0 = sdesc_kmajor_sw128(smem_u32(smem));
    int i = 0;
    for (; i < steps; i++) {
      const int s = i % ST, b = i % NBUF;
      if (!gemm_wait(&full[s], (i / ST) & 1, abort_flag, A.wait_ns) ||
          !gemm_wait(&tfree[b], ((i / NBUF) & 1) ^ 1, abort_flag, A.wait_ns))
        break;
      tc_fence_after();
      if (leader) {
        const uint64_t dw = d0 + (uint32_t)(s * (SB / 16)), dx = dw + M * 128 * kFp8Block / 16;
#pragma unroll
        for (int m = 0; m < M; m++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            mma_ss_e4m3(tmem + (b * M + m) * TN, dw + (uint32_t)(m * 128 * kFp8Block / 16) + 2u * j, dx + 2u * j,
                        idesc_e4m3(128, TN), j != 0);
        tc_commit(&tfull[b]);
        tc_commit(&empty[s]);
      }
      __syncwarp();
    }
    if (i < steps) {  // a wait expired: let the products in flight end before their tensor memory is given back
      if (leader) tc_commit(drain);
      mbar_wait_ns(drain, 0, kDrainWaitNs);
    }
  } else {
    const int wb = min(n0, A.rows - 1) / kFp8Block;
    const float* ws = A.w0.s + (int64_t)wb * A.nkb + kb_lo;
    const float* us = A.w1.s + (int64_t)wb * A.nkb + kb_lo;
    const float* xs = A.xs + (int64_t)min(lane, A.T - 1) * A.nkb + kb_lo;
    float* tab = table + warp * 2 * kSkinnyMaxT;  // [gate, up][token]
    const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
    uint64_t acc[M][TN / 2];
#pragma unroll
    for (int m = 0; m < M; m++)
#pragma unroll
      for (int c = 0; c < TN / 2; c++) acc[m][c] = 0;
    float xn = xs[0], wn = ws[0], un = GU ? us[0] : 0.f;
    bool ok = true;
    if (A.expire && warp == 0) ok = gemm_wait(never, 0, abort_flag, A.wait_ns);  // testing hook: this wait runs out
    for (int i = 0; ok && i < steps; i++) {
      const int b = i % NBUF;
      tab[lane] = xn * wn;
      if (GU) tab[kSkinnyMaxT + lane] = xn * un;
      bool far = __any_sync(0xffffffffu, not_normal(xn * wn) || (GU && not_normal(xn * un)));
      if (far) {
        far = false;
#pragma unroll
        for (int m = 0; m < M; m++) {
          const Scale f = scale_of(xn, m ? un : wn);
          tab[m * kSkinnyMaxT + lane] = f.small;
          tab[kBigs + m * kSkinnyMaxT + lane] = f.big;
          far |= f.big != 1.f;
        }
        far = __any_sync(0xffffffffu, far);
      }
      if (i + 1 < steps) {
        xn = xs[i + 1];
        wn = ws[i + 1];
        if (GU) un = us[i + 1];
      }
      __syncwarp();
      if (!(ok = gemm_wait(&tfull[b], (i / NBUF) & 1, abort_flag, A.wait_ns))) break;
      tc_fence_after();
      if (far)
#pragma unroll
        for (int m = 0; m < M; m++)
          scale_tmem<TN>(lanes + (b * M + m) * TN, [&](int c) { return tab[kBigs + m * kSkinnyMaxT + c]; });
#pragma unroll
      for (int m = 0; m < M; m++)
#pragma unroll
        for (int c0 = 0; c0 < TN; c0 += LD) {
          uint32_t r[LD];
          if constexpr (LD == 16) {
            tmem_ld16(lanes + (b * M + m) * TN + c0, r);
            tmem_wait_ld16(r);
          } else {
            tmem_ld32(lanes + (b * M + m) * TN + c0, r);
            tmem_wait_ld(r);
          }
#pragma unroll
          for (int c = 0; c < LD; c += 4) {
            const ulonglong2 sc = *reinterpret_cast<const ulonglong2*>(tab + m * kSkinnyMaxT + c0 + c);
            fma2(acc[m][(c0 + c) / 2], r[c], r[c + 1], sc.x);
            fma2(acc[m][(c0 + c) / 2 + 1], r[c + 2], r[c + 3], sc.y);
          }
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tfree[b]);
    }
    if (ok) {
      // All MMAs have read their operands: the ring takes the accumulators, [token][128 or 256 rows].
      float* dst = reinterpret_cast<float*>(smem) + 32 * warp + lane;
#pragma unroll
      for (int m = 0; m < M; m++)
#pragma unroll
        for (int c = 0; c < TN; c++)
          if (c < A.T) dst[c * (M * 128) + m * 128] = (c & 1) ? hi_of(acc[m][c / 2]) : lo_of(acc[m][c / 2]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, COLS);
  if (split > 1) {
    cluster_arrive();
    cluster_wait();
  }
  for (int t = rank + split * warp; t < A.T; t += split * (kSkinnyThreads / 32))
    finish_row<M, GU, GU>(A, reinterpret_cast<const float*>(smem) + (size_t)t * (M * 128), split, t, n0, lane);
  if (split > 1) {  // the peers have read this CTA's accumulators
    cluster_arrive();
    cluster_wait();
  }
}

cudaLaunchAttribute pdl() {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}
cudaLaunchAttribute cluster_of(int n) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = (unsigned)n;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}

// Lets the kernel use BYTES of dynamic shared memory, once per device (a second thread may repeat it).
template <auto KERN, size_t BYTES>
int allow_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -4;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return 0;
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)BYTES) != cudaSuccess) return -4;
  if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return 0;
}

// Map of a row-major e4m3 matrix, boxes of box_rows x 128 columns; columns and rows past the end read as zero.
int make_e4m3_map(CUtensorMap* map, const uint8_t* base, int rows, int cols, int box_rows) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return -4;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)cols};
  const cuuint32_t box[2] = {(cuuint32_t)kFp8Block, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : -4;
}

// CTAs that a tile's blocks are split over: the least time by the steps in a
// row, times the waves that the clusters need (a cluster lives inside one GPC,
// so 8 CTAs of one per SM fit 15 times, not 18, into 148 SMs). The two constants
// are estimates from a call's parts (start-up 0.7 us and first copies 0.9 us,
// two cluster barriers and the exchange, against 0.35 us a step), not fitted.
constexpr int kTileSteps = 6;   // start, drain and stores of a tile, in steps
constexpr int kSplitSteps = 6;  // the exchange between the CTAs of a cluster

template <auto KERN, size_t SMEM, int THREADS>
int pick_split(int64_t tiles, int nkb, int at_once) {
  static std::atomic<int> fit[64][kMaxSplit + 1];  // clusters that run at once; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -4;
  int best = 1;
  int64_t least = (tiles + at_once - 1) / at_once * (nkb + kTileSteps);
  for (int split = 2; split <= kMaxSplit && split <= nkb && tiles * split <= at_once; split++) {
    int n = dev < 64 ? fit[dev][split].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)split);
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = SMEM;
      cudaLaunchAttribute at[1] = {cluster_of(split)};
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&n, KERN, &cfg) != cudaSuccess) return -4;
      if (n < 1) n = -1;
      if (dev < 64) fit[dev][split].store(n, std::memory_order_relaxed);
    }
    if (n < 1) continue;
    const int64_t cost = (tiles + n - 1) / n * ((nkb + split - 1) / split + kTileSteps + kSplitSteps);
    if (cost < least) {
      least = cost;
      best = split;
    }
  }
  return best;
}

template <int BN, bool GU, bool PAIR>
int launch_gemm(const Fp8Args& a, int num_sms, cudaStream_t st) {
  constexpr int bm = PAIR ? 2 * kBM : kBM;
  const int tiles_m = (a.T + bm - 1) / bm, nb = GU ? 128 : BN, tiles_n = (a.rows + nb - 1) / nb;
  const int64_t tiles = (int64_t)tiles_m * tiles_n;
  if (tiles > 0x0fffffff) return -3;
  auto kern = k_fp8_gemm<BN, GU, PAIR>;
  static std::atomic<bool> checked{false};
  if (!checked.load(std::memory_order_relaxed)) {
    // the register split draws on what the launch takes: 5 x 96 for each lane of the five warpgroups
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return -4;
    if (fa.numRegs * (kGemmThreads / 128) != 4 * kEpiRegs + kLastRegs) return -3;
    checked.store(true);
  }
  if (allow_smem<k_fp8_gemm<BN, GU, PAIR>, kGemmSmem(BN, GU, PAIR)>()) return -4;
  const int split = PAIR ? 1 : pick_split<k_fp8_gemm<BN, GU, PAIR>, kGemmSmem(BN, GU, PAIR), kGemmThreads>(tiles, a.nkb, num_sms);
  if (split < 1) return split;
  CUtensorMap mx, m0, m1;
  if (make_e4m3_map(&mx, a.xq, a.T, a.cols, kBM) || make_e4m3_map(&m0, a.w0.q, a.rows, a.cols, 128)) return -4;
  if (GU ? make_e4m3_map(&m1, a.w1.q, a.rows, a.cols, 128) != 0 : (m1 = m0, false)) return -4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(PAIR        ? 2 * std::min<int64_t>(tiles, num_sms / 2)
                                : split > 1 ? tiles * split
                                            : std::min<int64_t>(tiles, num_sms)));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = kGemmSmem(BN, GU, PAIR);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {pdl(), cluster_of(PAIR ? 2 : split)};
  cfg.attrs = at;
  cfg.numAttrs = PAIR || split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, mx, m0, m1, a, tiles_m, (int)tiles, split) == cudaSuccess ? 0 : -4;
}

template <bool GU, int TN>
int launch_skinny(const Fp8Args& a, int num_sms, cudaStream_t st) {
  constexpr size_t smem = kSkSmem(GU, TN);
  const int tiles = (a.rows + 127) / 128;
  if (allow_smem<k_fp8_skinny<GU, TN>, smem>()) return -4;
  const int split = pick_split<k_fp8_skinny<GU, TN>, smem, kSkinnyThreads>(tiles, a.nkb, 2 * num_sms);
  if (split < 1) return split;
  CUtensorMap mx, m0, m1;
  if (make_e4m3_map(&mx, a.xq, a.T, a.cols, TN) || make_e4m3_map(&m0, a.w0.q, a.rows, a.cols, 128)) return -4;
  if (GU ? make_e4m3_map(&m1, a.w1.q, a.rows, a.cols, 128) != 0 : (m1 = m0, false)) return -4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(kSkinnyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {pdl(), cluster_of(split)};
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_skinny<GU, TN>, mx, m0, m1, a, split) == cudaSuccess ? 0 : -4;
}

}  // namespace

int launch_fp8_quantize(const uint16_t* x, int64_t stride, int T, int cols, uint8_t* q, float* s, cudaStream_t st,
                        int num_sms) {
  const int nkb = fp8_blocks(cols), items = T * nkb;
  const int per = kQuantThreads / kQuantLanes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((items + per - 1) / per, num_sms * kQuantBlocks));
  cfg.blockDim = dim3(kQuantThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1] = {pdl()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_fp8_quantize, x, stride, cols, nkb, FastDiv::of((uint32_t)nkb), items, q, s) ==
                 cudaSuccess
             ? 0
             : -4;
}

int launch_fp8_product(Fp8Args a, bool gate_up, cudaStream_t st, int num_sms) {
  a.wait_ns = wait_limit_ns();
  a.expire = waits_expire();
  if (a.T <= kSkinnyMaxT) {
    if (gate_up) return a.T <= 16 ? launch_skinny<true, 16>(a, num_sms, st) : launch_skinny<true, 32>(a, num_sms, st);
    return a.T <= 16 ? launch_skinny<false, 16>(a, num_sms, st) : launch_skinny<false, 32>(a, num_sms, st);
  }
  // Pairs of CTAs where their tiles occupy a third of the SMs or more. Pairs and
  // single CTAs at 4096 x 4096 weights: 512 tokens (32 tiles) 19.1 and 13.3 us,
  // 768 (48) 20.1 and 23.6, 1024 (64) 20.5 and 23.9; 4096 tokens of 1024 x 2048
  // (64) 13.5 and 14.5; gate_up of 2048 x 4096: 512 tokens (32) 20.1 and 17.3 us,
  // 768 (48) and 1024 (64) alike within 3%. The border is on the wrong side for
  // 640 to 768 tokens of the first (15%) and where rows of tokens are mostly
  // padding (300 tokens of 16384 x 1024: 16.0 and 13.0 us).
  const int cols = gate_up ? 128 : 256;
  const int64_t pairs = (int64_t)((a.T + 255) / 256) * ((a.rows + cols - 1) / cols);
  if (pairs * 3 >= num_sms)
    return gate_up ? launch_gemm<256, true, true>(a, num_sms, st) : launch_gemm<256, false, true>(a, num_sms, st);
  return gate_up ? launch_gemm<256, true, false>(a, num_sms, st) : launch_gemm<128, false, false>(a, num_sms, st);
}

int read_fp8_status(cudaStream_t st, int32_t* out) {
  if (cudaStreamSynchronize(st) != cudaSuccess) return -4;
  if (cudaMemcpyFromSymbol(out, g_fp8_status, 4) != cudaSuccess) return -4;
  const int32_t zero = 0;
  if (*out && cudaMemcpyToSymbol(g_fp8_status, &zero, 4) != cudaSuccess) return -4;
  return 0;
}

}  // namespace iqk
