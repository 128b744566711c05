// proj.cuh -- the matrix products around a sequence mixer, on tcgen05 tensor cores (sm_100a).
//
//     C[m][n] = sum_k A[m][k] B[n][k],      y = act(C + bias[n]) + residual[m][n]
//
// One kernel serves the projection (A = x, B = w) and its two gradients (dx: A = dz, B = w read
// along its other axis; dw: both read along the other axis): an operand whose rows run along m or
// n instead of k is staged as it lies and named so in the instruction descriptor.
//
// fp32 operands are split into three bf16 planes a = a0 + a1 + a2 (8 bits of the mantissa each),
// and C is the sum of the six products of planes i + j <= 2, smallest first; the three left out
// are below 2^-26 of a b.  (An operand below 2^-110 has planes among bf16's subnormals, which the
// tensor cores keep, or below the last of them, 2^-133, where its bits are lost.)  The planes of a
// k-block are three stages of the ring, from which the six products take theirs.  The tensor cores'
// accumulator truncates at every addition, which over thousands of k is a bias above fp32's own
// rounding: after each k-block the epilogue warps take the accumulator into registers, where the
// sum goes on with rounding to nearest (normwise error of a product over 4096 k: 1.2e-7, over
// 16384 k: 1.7e-7; fp32 FMAs: 1.1e-6 and 2.3e-6).  2048^3: 97 us (fp32 FMA units: 306).
//
// Tiles.  kCG = 2: a pair of CTAs works on 256 x 256 outputs with tcgen05.mma.cta_group::2, each
// holding 128 rows of A, 128 rows of B and 128 rows of the accumulator.  Each byte staged then
// feeds 128 products, twice what a single CTA's 128 x 128 tile gives; at the tensor cores' rate the
// pair draws 64 bytes per SM and cycle from L2, which L2 can serve, where 96 or 128 bytes starve
// it.  kCG = 1: 128 x kBN by one CTA, for problems with too few 256 x 256 tiles.  The tiles that do
// not fill a whole wave of workers are cut along k, and their fp32 partial products are summed, in
// order, by a second kernel.  Where all tiles are cut (small problems, a few tokens), the cuts of a
// tile are a cluster's CTAs (kJoin): each leaves its partial product in its shared memory and sums
// its share of the rows over the cluster, without a second kernel (8 x 4096 x 4096: 12.8 us with
// it).
//
// Persistent CTAs: warp 0 streams k-blocks of 64 through a ring of shared-memory stages with TMA
// (128-byte swizzle; zero fill at the ragged edges), warp 1 issues the MMAs into one of two
// accumulators in tensor memory, warps 2-9 drain the other: through shared memory, so that global
// rows are read and written in whole sectors.  Bound: the tensor pipe for large products, the
// bytes of w for a few rows.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace hyena {
namespace proj {

constexpr int kBK = 64;                        // k per stage: one 128-byte swizzled row
constexpr int kRows = 128;                     // rows of A (and of the accumulator) per CTA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kChunk = 32;                     // columns an epilogue warp stages at a time
constexpr int kStageOut = 32 * kChunk * 4;     // its staging bytes
constexpr int kMaxStages = 8;
constexpr unsigned int kTimeout = 1u;          // HYENA_DEVICE_TIMEOUT

enum Act { kNone = 0, kGelu = 1, kSilu = 2, kSigmoid = 3, kLogSigmoid = 4 };

// The six products of bf16 planes, smallest first, as (plane of A, plane of B).
constexpr int kProducts = 6;
__host__ __device__ constexpr int plane_a(int i) { return i == 1 ? 2 : i == 2 || i == 4 ? 1 : 0; }
__host__ __device__ constexpr int plane_b(int i) { return i == 0 ? 2 : i == 2 || i == 3 ? 1 : 0; }

template <int kCG, int kBN>
struct Tile {
  static constexpr int kM = kRows * kCG;               // of the whole tile
  static constexpr int kN = kBN;
  static constexpr int kBRows = kBN / kCG;             // rows of B per CTA
  static constexpr int kABytes = kRows * kBK * 2, kBBytes = kBRows * kBK * 2;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kFixed = kEpiWarps * kStageOut + 1024;
  static constexpr int kStages =
      (226 * 1024 - kFixed) / kStage < kMaxStages ? (226 * 1024 - kFixed) / kStage : kMaxStages;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static constexpr int kTmemCols = 2 * kBN < 32 ? 32 : 2 * kBN;  // two accumulators
};

struct Params {
  int M, N, kb;                 // outputs; k-blocks
  int tiles_m, tiles_n;
  int whole;                    // the first tiles, each one work
  int splits, kb_per_split;     // cuts of the other tiles' k-blocks
  int group_m;                  // tiles of m that run together (their w tiles stay in L2)
  const float *bias;            // [N] or null
  const void *residual;         // [M, N] or null
  void *y, *z;                  // [M, N]; z (before the activation) or null
  float *partial;               // [other tiles][splits][tile] when splits > 1
  int act;
  int tma;                      // whole tiles leave by TMA
  int bias_vec;                 // bias is 16-byte aligned
  int vec;                      // rows of y, z, residual are whole, aligned 16-byte vectors
  unsigned int *status;
  uint64_t wait_ns;             // limit of the waits between roles (bf16; 2 s but in tests)
  int fault;                    // test hook (enum Fault)
};
// 1: residuals are never requested; 2: the first accumulator is never announced; 3: the TMA warp of
// a pair's leader gives up after one stage
enum Fault { kNoFault = 0, kNoResidual = 1, kNoAccumulator = 2, kStagesEnd = 3 };

// ------------------------------------------------------------------------------- activations
// fp32 results take the accurate exp and division; a bf16 result rounds away what the fast ones
// lose (their sigmoid and silu end at z = -87.3, below 1e-36), and with the accurate division the
// epilogue of silu took longer than the product (8192 x 4096 x 4096: 340 us against 185).
template <typename T> __device__ __forceinline__ float exp_of(float x) { return __expf(x); }
template <> __device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }
template <typename T> __device__ __forceinline__ float ratio(float a, float b) { return __fdividef(a, b); }
template <> __device__ __forceinline__ float ratio<float>(float a, float b) { return a / b; }
template <typename T> __device__ __forceinline__ float sigmoid_of(float z) {
  return ratio<T>(1.0f, 1.0f + exp_of<T>(-z));
}

// 2 (1 - Phi(|z|)) = erfc(|z| / sqrt 2) from the exponential e = exp(-z^2 / 2), for bf16 results: e
// times a polynomial of degree 6 in t = 1 / (1 + 0.405 |z| / sqrt 2), without a constant term.  Its
// coefficients are a linear program's, which keeps the error below both 1e-7 and 2^-12 of the
// value for |z| < 13.5, past which e vanishes; fp32 roundings add 3e-7 near 1.  (An approximation
// held to an absolute error alone is a percent off at z = -8.)  Half the instructions of erff,
// which bound the epilogue of products over few k.
__device__ __forceinline__ float erfc_of(float z, float e) {
  const float t = __fdividef(1.0f, fmaf(0.28637823f, fabsf(z), 1.0f));
  float p = fmaf(-0.18832338f, t, 0.6349869f);
  p = fmaf(p, t, -0.26931491f);
  p = fmaf(p, t, 0.4052876f);
  p = fmaf(p, t, 0.18515244f);
  p = fmaf(p, t, 0.23221135f);
  return p * t * e;
}
// Phi(z) for fp32 results: erfc, since 1 + erf rounds away what is left of it below zero.
__device__ __forceinline__ float phi_of(float z) { return 0.5f * erfcf(z * -0.70710678f); }
template <typename T>
__device__ __forceinline__ float gelu_of(float z) {
  if constexpr (sizeof(T) == 4) return z * phi_of(z);
  // z times Phi, which is 1 at +inf (z less a part of z would be inf - inf times 0 there)
  const float tail = 0.5f * erfc_of(z, __expf(-0.5f * z * z));  // 1 - Phi(|z|)
  return z * (z > 0.0f ? 1.0f - tail : tail);
}
template <typename T>
__device__ __forceinline__ float gelu_slope(float z) {
  const float e = exp_of<T>(-0.5f * z * z);
  if constexpr (sizeof(T) == 4) return fmaf(z * 0.39894228f, e, phi_of(z));
  const float tail = 0.5f * erfc_of(z, e);
  return fmaf(z * 0.39894228f, e, z > 0.0f ? 1.0f - tail : tail);
}

// log(1 + e) for 0 <= e <= 1; for bf16 results the fast logarithm, and near 0, where 1 + e rounds
// most of e away, three terms of the series (within 2^-20 of the value at e = 2^-6).
template <typename T>
__device__ __forceinline__ float log1p_of(float e) {
  if constexpr (sizeof(T) == 4) return log1pf(e);
  return e < 0.015625f ? e * fmaf(e, fmaf(e, 0.33333333f, -0.5f), 1.0f) : __logf(1.0f + e);
}

template <typename T, int kAct>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (kAct == kGelu) return gelu_of<T>(z);
  if constexpr (kAct == kSilu) return ratio<T>(z, 1.0f + exp_of<T>(-z));
  if constexpr (kAct == kSigmoid) return sigmoid_of<T>(z);
  if constexpr (kAct == kLogSigmoid) return fminf(z, 0.0f) - log1p_of<T>(exp_of<T>(-fabsf(z)));
  return z;
}

template <typename T, int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (kAct == kGelu) return gelu_slope<T>(z);
  if constexpr (kAct == kSilu) {
    const float p = sigmoid_of<T>(z);
    return p * (1.0f + z * (1.0f - p));
  }
  if constexpr (kAct == kSigmoid) {  // p (1 - p), where 1 - p of a p near 1 has few bits left
    const float e = exp_of<T>(-fabsf(z)), d = 1.0f + e;
    return ratio<T>(e, d * d);
  }
  if constexpr (kAct == kLogSigmoid) return sigmoid_of<T>(-z);
  return 1.0f;
}

// f(integral constant of the activation), one branch for all the elements that f handles.
template <typename F>
__device__ __forceinline__ void with_act(int act, F &&f) {
  switch (act) {
    case kGelu: f(std::integral_constant<int, kGelu>()); break;
    case kSilu: f(std::integral_constant<int, kSilu>()); break;
    case kSigmoid: f(std::integral_constant<int, kSigmoid>()); break;
    case kLogSigmoid: f(std::integral_constant<int, kLogSigmoid>()); break;
    default: f(std::integral_constant<int, kNone>());
  }
}

// ------------------------------------------------------------------------------- elements
template <typename T, int n> struct alignas(sizeof(T) * n) VecOf { T e[n]; };
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, float *o) { *o = x; }

// Residuals are read, and outputs written, once: first out of L2, where tiles of x and w are read
// many times over.
template <typename T, int n>
__device__ __forceinline__ VecOf<T, n> load_once(const T *p) {
  VecOf<T, n> v;
  if constexpr (sizeof(v) == 16)
    *reinterpret_cast<uint4 *>(&v) = __ldcs(reinterpret_cast<const uint4 *>(p));
  else
    *reinterpret_cast<uint2 *>(&v) = __ldcs(reinterpret_cast<const uint2 *>(p));
  return v;
}
template <typename T, int n>
__device__ __forceinline__ void store_once(T *p, const VecOf<T, n> &v) {
  if constexpr (sizeof(v) == 16)
    __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&v));
  else
    __stcs(reinterpret_cast<uint2 *>(p), *reinterpret_cast<const uint2 *>(&v));
}

// Activation, residual and the one rounding of n neighbouring outputs of a row; z is the product
// with its bias.
template <typename T, int n>
__device__ __forceinline__ void finish(const Params &p, const float (&z)[n], int64_t row, int col) {
  constexpr int V = 16 / static_cast<int>(sizeof(T)) < n ? 16 / static_cast<int>(sizeof(T)) : n;
  const int64_t at = row * p.N + col;
  float y[n];
  with_act(p.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] = act_of<T, decltype(act)::value>(z[i]);
  });
  if (p.vec && col + n <= p.N) {
#pragma unroll
    for (int i0 = 0; i0 < n; i0 += V) {
      VecOf<T, V> r, o;
      if (p.residual) {
        r = load_once<T, V>(static_cast<const T *>(p.residual) + at + i0);
#pragma unroll
        for (int i = 0; i < V; ++i) y[i0 + i] += to_f(r.e[i]);
      }
      if (p.z) {
#pragma unroll
        for (int i = 0; i < V; ++i) from_f(z[i0 + i], &o.e[i]);
        store_once<T, V>(static_cast<T *>(p.z) + at + i0, o);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) from_f(y[i0 + i], &o.e[i]);
      store_once<T, V>(static_cast<T *>(p.y) + at + i0, o);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      if (col + i >= p.N) break;
      if (p.residual) y[i] += to_f(static_cast<const T *>(p.residual)[at + i]);
      if (p.z) from_f(z[i], static_cast<T *>(p.z) + at + i);
      from_f(y[i], static_cast<T *>(p.y) + at + i);
    }
  }
}

// ------------------------------------------------------------------------------- pairs of CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(p));
  return p != 0;
}
// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void put_in_cta(int *p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
template <int kCG>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint32_t bar, int x,
                                          int y, int plane) {
  if constexpr (kCG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(plane)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile"
        ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(plane)
        : "memory");
}
// One MMA; the descriptors' low words (addresses) change from one to the next, the high do not.
template <int kCG>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                    uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kCG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` (of every CTA of the group) when the MMAs issued so far are done.
template <int kCG>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (kCG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
template <int kCG>
__device__ __forceinline__ void tmem_get(uint32_t *dst, uint32_t cols) {
  if constexpr (kCG == 2)
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
        "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst)),
        "r"(cols)
        : "memory");
  else
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
        "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::"r"(smem_u32(dst)),
        "r"(cols)
        : "memory");
}
template <int kCG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if constexpr (kCG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                 : "memory");
  else
    tmem_dealloc(base, cols);
}

// Instruction descriptor: bf16 operands, fp32 accumulator, major-ness of each (1: rows along m/n).
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return umma_idesc_f16_f32_mn(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

// ------------------------------------------------------------------------------- work
struct Work {
  int m, n, kb0, kb1;  // tile coordinates; k-blocks [kb0, kb1)
  int part;            // index of its partial product, or -1
};
__device__ __forceinline__ void tile_at(const Params &p, int t, int *m, int *n) {
  const int per = p.group_m * p.tiles_n, g = t / per, r = t % per;
  const int gm = min(p.group_m, p.tiles_m - g * p.group_m);
  *m = g * p.group_m + r % gm;
  *n = r / gm;
}
__device__ __forceinline__ int work_count(const Params &p) {
  return p.whole + (p.tiles_m * p.tiles_n - p.whole) * p.splits;
}
__device__ __forceinline__ Work work_at(const Params &p, int w) {
  Work k;
  const int rest = p.tiles_m * p.tiles_n - p.whole;
  int tile = w;
  k.kb0 = 0;
  k.kb1 = p.kb;
  k.part = -1;
  if (w >= p.whole && p.splits > 1) {  // a cut of all the other tiles, then the next cut
    const int r = w - p.whole, split = r / rest;
    tile = p.whole + r % rest;
    k.kb0 = split * p.kb_per_split;
    k.kb1 = min(k.kb0 + p.kb_per_split, p.kb);
    k.part = (r % rest) * p.splits + split;
  }
  tile_at(p, tile, &k.m, &k.n);
  return k;
}

// ------------------------------------------------------------------------------- the product
// kAMn / kBMn: the operand's rows run along m / n (its tensor map is [k][m]), else along k.
template <typename T, int kCG, int kBN, bool kAMn, bool kBMn, bool kJoin>
__global__ void __launch_bounds__(kThreads, 1)
    proj_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mz,
                const __grid_constant__ CUtensorMap mr, const Params p) {
  using L = Tile<kCG, kBN>;
  constexpr bool kPromote = sizeof(T) == 4;
  constexpr int kPlanes = kPromote ? 3 : 1;                // stages of a k-block
  constexpr int kRing = L::kStages / kPlanes * kPlanes;  // stages in use
  static_assert(!kPromote || kCG == 1, "the sums of a pair's tile do not fit the registers");
  static_assert(!kJoin || kCG == 1, "a cluster is a pair or a tile's cuts");
  extern __shared__ uint8_t dynamic[];
  __shared__ uint64_t full[L::kStages], empty[L::kStages], acc_full[2], acc_empty[2];
  __shared__ uint64_t res_full[kEpiWarps];
  __shared__ uint32_t tmem_at;
  __shared__ int abort;
  __shared__ int issued, peer_abort, peer_issued;  // issued: stages with copies under way or landed
  uint8_t *stages = dynamic + (1024 - smem_u32(dynamic) % 1024) % 1024;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = kCG == 2 ? cluster_rank() : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps * kCG);
    }
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(&res_full[i], 1);
    abort = 0;
    peer_abort = peer_issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_get<kCG>(&tmem_at, L::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  if (kCG == 2) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_at;
  // kJoin: one work for each CTA, cut by cut of one tile in a cluster
  const int works = work_count(p), tiles = p.tiles_m * p.tiles_n;
  const int first = kJoin ? static_cast<int>(blockIdx.x) % p.splits * tiles +
                                static_cast<int>(blockIdx.x) / p.splits
                          : static_cast<int>(blockIdx.x) / kCG;
  const int step = kJoin ? works : static_cast<int>(gridDim.x) / kCG;
  griddep_launch_dependents();
  griddep_wait();

  // A wait of the whole warp, with one answer for all of it.
  const auto wait = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu,
                      mbar_wait(bar, parity, &abort, p.status, kTimeout,
                                kPromote ? kWaitTimeoutNs : p.wait_ns)) != 0;
  };
  // The TMA and MMA warps run their loops as a whole and only the instruction itself in one lane:
  // descriptors and coordinates then stay in uniform registers.  With the loops inside one lane,
  // moving every operand there took 0.3 us per k-block (a cuBLAS block: 0.08).
  if (warp == 0) {
    // --------------------------------------------------------------------------- TMA
    const bool lead = elect_one();
    int it = 0, st = 0;
    uint32_t freed = 1;  // parity of the stage's last release; the first round waits for none
    bool ok = true;
    const uint32_t full0 = kCG == 2 ? in_cta(&full[0], 0) : smem_u32(&full[0]);
    for (int w = first; w < works && ok; w += step) {
      const Work k = work_at(p, w);
      const int m0 = k.m * L::kM + static_cast<int>(rank) * kRows;
      const int n0 = k.n * L::kN + static_cast<int>(rank) * L::kBRows;
      for (int i = k.kb0 * kPlanes; i < k.kb1 * kPlanes; ++i, ++it) {
        if (it >= kRing && !wait(&empty[st], freed)) {
          ok = false;
          break;
        }
        if (kCG == 2 && p.fault == kStagesEnd && rank == 0 && it == 1) {
          abort = 1;
          if (lead) atomicOr(p.status, kTimeout);
          ok = false;
          break;
        }
        const int plane = i % kPlanes, k0 = i / kPlanes * kBK;
        uint8_t *a = stages + st * L::kStage, *b = a + L::kABytes;
        const uint32_t bar = full0 + 8 * st;
        if (lead) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st], kCG * L::kStage);
          if (kAMn) {
#pragma unroll
            for (int h = 0; h < kRows / 64; ++h)
              load_tile<kCG>(a + h * 8192, &ma, bar, m0 + h * 64, k0, plane);
          } else {
            load_tile<kCG>(a, &ma, bar, k0, m0, plane);
          }
          if (kBMn) {
#pragma unroll
            for (int h = 0; h < L::kBRows / 64; ++h)
              load_tile<kCG>(b + h * 8192, &mb, bar, n0 + h * 64, k0, plane);
          } else {
            load_tile<kCG>(b, &mb, bar, k0, n0, plane);
          }
        }
        if (++st == kRing) {
          st = 0;
          freed ^= 1;
        }
      }
    }
    // Before the CTA ends every copy has landed and every release of a stage has arrived.  In
    // the leader `full` covers both CTAs' copies.
    for (int j = it > kRing ? it - kRing : 0; j < it; ++j) {
      const int s = j % kRing, parity = (j / kRing) & 1;
      int no_abort = 0;
      if (!wait(&empty[s], parity) && rank == 0)
        mbar_wait(&full[s], parity, &no_abort, p.status, kTimeout);
    }
    if (lane == 0) issued = it;
  } else if (warp == 1) {
    if (rank == 0) {
      // ------------------------------------------------------------------------- MMA
      constexpr uint32_t id = idesc_bf16(L::kM, L::kN, kAMn, kBMn);
      constexpr uint32_t kStepA = (kAMn ? 16 * 128 : 32) >> 4, kStepB = (kBMn ? 16 * 128 : 32) >> 4;
      const bool lead = elect_one();
      const uint32_t s0 = smem_u32(stages);
      const uint64_t da0 = umma_smem_desc(s0, kAMn ? 8192 : 16, 1024, 2);
      const uint64_t db0 = umma_smem_desc(s0 + L::kABytes, kBMn ? 8192 : 16, 1024, 2);
      const uint32_t a_hi = static_cast<uint32_t>(da0 >> 32), b_hi = static_cast<uint32_t>(db0 >> 32);
      uint32_t a_lo = static_cast<uint32_t>(da0), b_lo = static_cast<uint32_t>(db0);
      int it = 0, n = 0, st = 0;  // stages taken; accumulators filled; stage
      uint32_t filled = 0;        // parity of the stage's next fill
      bool ok = true;
      for (int w = first; w < works && ok; w += step) {
        const Work k = work_at(p, w);
        for (int kb = k.kb0; kb < k.kb1 && ok; ++n) {
          const int acc = n & 1, end = kPromote ? kb + 1 : k.kb1;
          if (n >= 2 && !wait(&acc_empty[acc], (n / 2 - 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d = tmem + acc * kBN;
          for (uint32_t more = 0; kb < end; ++kb, it += kPlanes) {
#pragma unroll
            for (int q = 0; q < kPlanes; ++q) ok = ok && wait(&full[st + q], filled);
            if (!ok) break;
            tc_fence_after_sync();
            if (lead) {
#pragma unroll
              for (int q = 0; q < (kPromote ? kProducts : 1); ++q) {
                constexpr uint32_t kUnits = L::kStage >> 4;
                const uint32_t a = a_lo + (kPromote ? plane_a(q) * kUnits : 0);
                const uint32_t b = b_lo + (kPromote ? plane_b(q) * kUnits : 0);
#pragma unroll
                for (int s = 0; s < kBK / 16; ++s)
                  mma<kCG>(d, a + s * kStepA, a_hi, b + s * kStepB, b_hi, id,
                           q > 0 || s > 0 ? 1u : more);
              }
#pragma unroll
              for (int q = 0; q < kPlanes; ++q) commit<kCG>(&empty[st + q]);
            }
            more = 1;
            a_lo += kPlanes * (L::kStage >> 4);
            b_lo += kPlanes * (L::kStage >> 4);
            st += kPlanes;
            if (st == kRing) {
              st = 0;
              filled ^= 1;
              a_lo = static_cast<uint32_t>(da0);
              b_lo = static_cast<uint32_t>(db0);
            }
          }
          if (ok && lead && (kPromote || p.fault != kNoAccumulator || n > 0))
            commit<kCG>(&acc_full[acc]);
          __syncwarp();
        }
      }
      // The MMAs issued are done before the CTA ends, also where another warp gives up after this
      // one has issued its last.
      int no_abort = 0;
      for (int j = it > kRing ? it - kRing : 0; j < it; ++j)
        mbar_wait(&empty[j % kRing], (j / kRing) & 1, &no_abort, p.status, kTimeout);
    }
  } else {
    // --------------------------------------------------------------------------- epilogue
    const int quad = warp % 4;             // the 32 lanes of tensor memory that this warp may read
    const int col0 = (warp - 2) / 4 * (kBN / 2);  // its half of the columns
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + col0;
    float *out = reinterpret_cast<float *>(stages + L::kStages * L::kStage + (warp - 2) * kStageOut);
    const auto release = [&](int acc) {  // the accumulator is in registers: the next may start
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (kCG == 2)
          arrive_at(in_cta(&acc_empty[acc], 0));
        else
          mbar_arrive(&acc_empty[acc]);
      }
    };
    // Whole bf16 tiles leave by TMA: a chunk of 32 x 32 outputs is finished in registers (a lane
    // has a row), written to one of two buffers in the layout of the 64-byte swizzle and stored from
    // there; a residual comes into the buffer the same way, a chunk ahead, and is overwritten in
    // place.  (Through fp32 staging and plain stores the epilogue took three times as long, which
    // is what products over few k are bound by.)
    uint8_t *bufs = reinterpret_cast<uint8_t *>(out);
    uint64_t *res_bar = &res_full[warp - 2];
    [[maybe_unused]] uint64_t once = 0;  // L2 policy of what is read or written once
    [[maybe_unused]] uint32_t writes = 0, res_asked = 0, res_seen = 0;  // res_*: residual chunks
    if constexpr (!kPromote)
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
    // Requests the residual of the chunk at column c0 of work k into the buffer of write `at`; the
    // stores so far have read their buffers.
    const auto request = [&](const Work &k, int c0, uint32_t at) {
      if (p.fault == kNoResidual) return;
      ++res_asked;
      if (lane == 0) {
        mbar_arrive_expect_tx(res_bar, 2048);
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(
                smem_u32(bufs + (at & 1) * 2048)),
            "l"(reinterpret_cast<uint64_t>(&mr)), "r"(smem_u32(res_bar)),
            "r"(k.n * L::kN + col0 + c0),
            "r"(k.m * L::kM + static_cast<int>(rank) * kRows + quad * 32), "r"(0), "l"(once)
            : "memory");
      }
    };
    // Stores the rows that the lanes hold at (row0, col) from the buffer of the next write.
    const auto store = [&](const CUtensorMap *map, const float (&v)[32], int row0, int col) {
      uint8_t *buf = bufs + (writes & 1) * 2048;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
          o[e] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (col < p.N && row0 < p.M)
          asm volatile(
              "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group.L2::cache_hint"
              " [%0, {%2, %3, %4}], [%1], %5;" ::"l"(reinterpret_cast<uint64_t>(map)),
              "r"(smem_u32(buf)), "r"(col), "r"(row0), "r"(0), "l"(once)
              : "memory");
        bulk_commit_group();
      }
      ++writes;
    };
    const bool ahead = p.tma && p.residual;  // residuals are requested a chunk ahead
    if (!kPromote && ahead && first < works) {
      const Work k = work_at(p, first);
      if (k.part < 0) request(k, 0, 0);
    }
    int n = 0;
    bool ok = true;
    for (int w = first; w < works && ok; w += step) {
      const Work k = work_at(p, w);
      const int row0 = k.m * L::kM + static_cast<int>(rank) * kRows + quad * 32;
      [[maybe_unused]] float sum[kPromote ? kBN / 2 : 1];
      if constexpr (kPromote) {
#pragma unroll
        for (int c = 0; c < kBN / 2; ++c) sum[c] = 0.0f;
        for (int kb = k.kb0; kb < k.kb1 && ok; ++kb, ++n) {
          const int acc = n & 1;
          ok = wait(&acc_full[acc], (n / 2) & 1);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int c0 = 0; c0 < kBN / 2; c0 += 32) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(lanes + acc * kBN + c0, r);
            tmem_wait_ld();
            reg_fence(r);
#pragma unroll
            for (int c = 0; c < 32; ++c) sum[c0 + c] += __uint_as_float(r[c]);
          }
          release(acc);
        }
      } else {
        ok = wait(&acc_full[n & 1], (n / 2) & 1);
        tc_fence_after_sync();
      }
      if (!ok) break;
      if constexpr (kJoin) {
        // the partial product, in the ring's memory (its last MMA is done): row `quad * 32 + lane`,
        // 16-byte pieces swizzled by the row
        float *part = reinterpret_cast<float *>(stages) + (quad * 32 + lane) * kBN + col0;
#pragma unroll
        for (int c0 = 0; c0 < kBN / 2; c0 += 32) {
          float v[32];
          if constexpr (kPromote) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = sum[c0 + e];
          } else {
            uint32_t r[32];
            tmem_ld_32x32b_x32(lanes + (n & 1) * kBN + c0, r);
            tmem_wait_ld();
            reg_fence(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4 *>(part + c0 + ((j ^ (lane & 7)) * 4)) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
        if (!kPromote) ++n;
        continue;
      }
      if constexpr (!kPromote) {
        if (p.tma && k.part < 0) {
#pragma unroll 1
          for (int c0 = 0; c0 < kBN / 2; c0 += kChunk) {
            const bool last = c0 + kChunk >= kBN / 2;
            const int col = k.n * L::kN + col0 + c0;
            float v[32];
            {
              uint32_t r[32];
              tmem_ld_32x32b_x32(lanes + (n & 1) * kBN + c0, r);
              tmem_wait_ld();
              reg_fence(r);
              if (last) release(n & 1);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
            }
            if (p.bias) {  // N is a multiple of 8: pieces of 4 are inside or outside
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                if (col + e >= p.N) break;
                if (p.bias_vec) {
                  const float4 b = *reinterpret_cast<const float4 *>(p.bias + col + e);
                  v[e] += b.x, v[e + 1] += b.y, v[e + 2] += b.z, v[e + 3] += b.w;
                } else {
#pragma unroll
                  for (int i = 0; i < 4; ++i) v[e + i] += p.bias[col + e + i];
                }
              }
            }
            if (p.z) {  // (never with a residual here: the buffers are the stores' alone)
              if (lane == 0) bulk_wait_group_read<1>();
              __syncwarp();
              store(&mz, v, row0, col);
            }
            with_act(p.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = act_of<T, decltype(act)::value>(v[e]);
            });
            if (p.residual) {
              ok = wait(res_bar, res_seen & 1);
              if (!ok) break;  // no further request on this barrier: its phase is still open
              ++res_seen;
              const uint8_t *buf = bufs + (writes & 1) * 2048;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 u =
                    *reinterpret_cast<const uint4 *>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16));
                const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  v[8 * j + 2 * e] += __uint_as_float(word[e] << 16);
                  v[8 * j + 2 * e + 1] += __uint_as_float(word[e] & 0xffff0000u);
                }
              }
              if (lane == 0) bulk_wait_group_read<0>();
              __syncwarp();
              if (!last) {
                request(k, c0 + kChunk, writes + 1);
              } else if (w + step < works) {
                const Work next = work_at(p, w + step);
                if (next.part < 0) request(next, 0, writes + 1);
              }
            } else {
              if (lane == 0) bulk_wait_group_read<1>();
              __syncwarp();
            }
            store(&my, v, row0, col);
          }
          ++n;
          continue;
        }
        // the staging below takes both buffers
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
      }
      const bool wide = kPromote && p.vec && k.part < 0;
#pragma unroll(kPromote ? kBN / 2 / kChunk : 1)
      for (int c0 = 0; c0 < kBN / 2; c0 += kChunk) {
        // phase 2: lane -> rows 8 i + lane / 4, columns col .. col + 7 of the warp's 32 rows
        const int in_tile = col0 + c0 + (lane % 4) * 8, col = k.n * L::kN + in_tile;
        const bool last = c0 + kChunk >= kBN / 2;
        constexpr int V = 16 / static_cast<int>(sizeof(T));
        const int sub = lane / 4;
        [[maybe_unused]] VecOf<T, 8> res[4];  // requested before the accumulator is touched
        if (wide && p.residual) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 8; h += V)
              if (row0 + 8 * i + sub < p.M && col + h < p.N)
                *reinterpret_cast<VecOf<T, V> *>(&res[i].e[h]) =
                    load_once<T, V>(static_cast<const T *>(p.residual) +
                                    static_cast<int64_t>(row0 + 8 * i + sub) * p.N + col + h);
        }
        float bias[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          bias[e] = p.bias && k.part < 0 && col + e < p.N ? p.bias[col + e] : 0.0f;
        // phase 1: row `lane` into shared memory, in 16-byte pieces swizzled by the row
        uint32_t r[32];
        if constexpr (kPromote) {
#pragma unroll
          for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(sum[c0 + c]);
        } else {
          tmem_ld_32x32b_x32(lanes + (n & 1) * kBN + c0, r);
          tmem_wait_ld();
          reg_fence(r);
          if (last) release(n & 1);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4 *>(out + lane * kChunk + ((j ^ (lane & 7)) * 4)) =
              make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        __syncwarp();
        const auto staged = [&](int i, float (&c)[8]) {
          const int rr = 8 * i + sub, j = 2 * (lane % 4);
          const float *src = out + rr * kChunk;
          const float4 u = *reinterpret_cast<const float4 *>(src + ((j ^ (rr & 7)) * 4));
          const float4 v = *reinterpret_cast<const float4 *>(src + (((j + 1) ^ (rr & 7)) * 4));
          c[0] = u.x + bias[0], c[1] = u.y + bias[1], c[2] = u.z + bias[2], c[3] = u.w + bias[3];
          c[4] = v.x + bias[4], c[5] = v.y + bias[5], c[6] = v.z + bias[6], c[7] = v.w + bias[7];
        };
        if (kPromote && wide) {
          with_act(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float c[8];
              staged(i, c);
              const int row = row0 + 8 * i + sub;
              if (row >= p.M) continue;
              const int64_t at = static_cast<int64_t>(row) * p.N + col;
#pragma unroll
              for (int h = 0; h < 8; h += V) {
                if (col + h >= p.N) break;
                VecOf<T, V> o;
                if (p.z) {
#pragma unroll
                  for (int e = 0; e < V; ++e) from_f(c[h + e], &o.e[e]);
                  store_once<T, V>(static_cast<T *>(p.z) + at + h, o);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                  float y = act_of<T, decltype(act)::value>(c[h + e]);
                  if (p.residual) y += to_f(res[i].e[h + e]);
                  from_f(y, &o.e[e]);
                }
                store_once<T, V>(static_cast<T *>(p.y) + at + h, o);
              }
            }
          });
        } else {
          // rows that are no multiple of 16 bytes, and partial products: lane -> column, row by row,
          // eight rows' residuals at a time
          const int at = k.n * L::kN + col0 + c0 + lane;
          const bool inside = at < p.N;
          const float b = p.bias && k.part < 0 && inside ? p.bias[at] : 0.0f;
          const T *res = static_cast<const T *>(p.residual);
#pragma unroll 1
          for (int r0 = 0; r0 < 32; r0 += 8) {
            float add[8], v[8];
            const int64_t first_at = static_cast<int64_t>(row0 + r0) * p.N + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              add[i] = k.part < 0 && res && inside && row0 + r0 + i < p.M
                           ? to_f(res[first_at + static_cast<int64_t>(i) * p.N])
                           : 0.0f;
              v[i] = b + out[(r0 + i) * kChunk + (((lane >> 2) ^ i) * 4) + (lane & 3)];
            }
            if (k.part >= 0) {  // whole tiles of fp32: no care at the ragged edge
              float *to = p.partial +
                          (static_cast<int64_t>(k.part) * L::kM + static_cast<int>(rank) * kRows +
                           quad * 32 + r0) * kBN + col0 + c0 + lane;
#pragma unroll
              for (int i = 0; i < 8; ++i) to[i * kBN] = v[i];
              continue;
            }
            float y[8];
            with_act(p.act, [&](auto act) {
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = act_of<T, decltype(act)::value>(v[i]) + add[i];
            });
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (!inside || row0 + r0 + i >= p.M) continue;
              const int64_t to = first_at + static_cast<int64_t>(i) * p.N;
              if (p.z) from_f(v[i], static_cast<T *>(p.z) + to);
              from_f(y[i], static_cast<T *>(p.y) + to);
            }
          }
        }
        __syncwarp();
      }
      if (!kPromote) ++n;
    }
    if constexpr (!kPromote) {
      if (lane == 0) {
        bulk_wait_group<0>();
        // a residual requested for a chunk that a failed wait kept from being read
        int no_abort = 0;
        if (res_asked != res_seen) mbar_wait(res_bar, res_seen & 1, &no_abort, p.status, kTimeout);
      }
      __syncwarp();
    }
  }
  // Both CTAs' MMAs read each other's shared memory and signal each other's barriers.
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (kCG == 2) {
    if (threadIdx.x == 0 && abort) {
      put_in_cta(&peer_issued, rank ^ 1, issued);
      put_in_cta(&peer_abort, rank ^ 1, 1);
    }
    cluster_sync();
    if (abort || peer_abort) {  // in both CTAs
      // The other CTA's copies for stages that the leader gave up before: their bytes count on the
      // leader's barriers, which it arms for them alone.
      if (rank == 0 && warp == 0) {
        int no_abort = 0;
        for (int j = issued; j < peer_issued; ++j) {
          if (lane == 0) mbar_arrive_expect_tx(&full[j % kRing], L::kStage);
          __syncwarp();
          mbar_wait(&full[j % kRing], (j / kRing) & 1, &no_abort, p.status, kTimeout);
        }
      }
      __syncwarp();
      cluster_sync();
    }
  }
  if constexpr (kJoin) {
    cluster_sync();  // every cut's partial product is there
    if (warp >= 2 && !abort) {
      const Work k = work_at(p, first);
      const int cut = static_cast<int>(cluster_rank()), m0 = k.m * kRows;
      const int rows = min(kRows, p.M - m0);  // those in range are shared out
      const int r0 = rows * cut / p.splits, r1 = rows * (cut + 1) / p.splits;
      constexpr int kQuads = kBN / 4;
      const uint32_t base = smem_u32(stages);
      constexpr int kBatch = 4;  // pieces in flight per thread
      const int n = (r1 - r0) * kQuads, step_i = 32 * kEpiWarps;
      for (int i0 = threadIdx.x - 64; i0 < n; i0 += kBatch * step_i) {
        float c[kBatch][4] = {};
        for (int s = 0; s < p.splits; ++s) {
          uint32_t peer;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(base), "r"(s));
          float4 v[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int i = min(i0 + b * step_i, n - 1), r = r0 + i / kQuads, q = i % kQuads;
            // pieces are swizzled within groups of 8
            const uint32_t at = peer + (r * kBN + ((q & ~7) | ((q ^ r) & 7)) * 4) * 4;
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[b].x), "=f"(v[b].y), "=f"(v[b].z), "=f"(v[b].w)
                         : "r"(at));
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
            c[b][0] += v[b].x, c[b][1] += v[b].y, c[b][2] += v[b].z, c[b][3] += v[b].w;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b * step_i, r = r0 + i / kQuads, col = k.n * kBN + i % kQuads * 4;
          if (i >= n || col >= p.N) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) c[b][e] += p.bias && col + e < p.N ? p.bias[col + e] : 0.0f;
          finish<T, 4>(p, c[b], m0 + r, col);
        }
      }
    }
    __syncwarp();    // the barrier wants whole warps, and the lanes' shares of the rows may differ
    cluster_sync();  // no CTA leaves while others read its product
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_free<kCG>(tmem, L::kTmemCols);
  }
}

// The sums of the cut tiles' partial products, in order, and their epilogue: a tile per blockIdx.y
// (and every gridDim.y-th after it), four columns of a row per thread.
template <typename T, int kM, int kN>
__global__ void __launch_bounds__(256) proj_join_kernel(const Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int rest = p.tiles_m * p.tiles_n - p.whole;
  for (int tile = blockIdx.y; tile < rest; tile += gridDim.y) {
    int tm, tn;
    tile_at(p, p.whole + tile, &tm, &tn);
    // rows of a tile that can be in range at all: a product of few rows fills little of its tiles
    const int rows = min(kM, p.M - tm * kM);
    const float *part = p.partial + static_cast<int64_t>(tile) * p.splits * (kM * kN);
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < rows * (kN / 4);
         i += gridDim.x * blockDim.x) {
      const int r = i / (kN / 4), c4 = i % (kN / 4) * 4, col = tn * kN + c4;
      if (col >= p.N) continue;
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      const float *from = part + r * kN + c4;
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) {
        const float4 v = *reinterpret_cast<const float4 *>(from + static_cast<int64_t>(s) * (kM * kN));
        c[0] += v.x, c[1] += v.y, c[2] += v.z, c[3] += v.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] += p.bias && col + e < p.N ? p.bias[col + e] : 0.0f;
      finish<T, 4>(p, c, static_cast<int64_t>(tm) * kM + r, col);
    }
  }
}

// ------------------------------------------------------------------------------- operands
// Eight values as bf16 planes, each the nearest to what the planes before leave; one plane is the
// value rounded.  Of three, the first goes towards zero where the nearest would overflow, and values
// that are not finite stay in it (times a zero plane of their partner they give NaN).
template <int kPlanes>
__device__ __forceinline__ void planes_of(const float (&v)[8], VecOf<__nv_bfloat16, 8> (&o)[kPlanes]) {
  if constexpr (kPlanes == 1) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      *reinterpret_cast<__nv_bfloat162 *>(&o[0].e[e]) = __floats2bfloat162_rn(v[e], v[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = v[e];
      const bool finite = isfinite(x);
#pragma unroll
      for (int q = 0; q < kPlanes; ++q) {
        __nv_bfloat16 b = __float2bfloat16_rn(x);
        if (q == 0 && finite && isinf(__bfloat162float(b))) b = __float2bfloat16_rz(x);
        o[q].e[e] = b;
        x = finite ? x - __bfloat162float(b) : 0.0f;
      }
    }
  }
}

// Rows of `cols` elements as rows of `ld` bf16 (a multiple of 8, zero past cols): one plane for
// bf16, three for fp32.  Eight elements of a row per thread; one launch for up to two operands of
// the same row length.
template <typename T>
struct Pack {
  const T *src;
  __nv_bfloat16 *dst;
  int64_t rows;
};
template <typename T>
__global__ void __launch_bounds__(256)
    proj_pack_kernel(const Pack<T> a, const Pack<T> b, int cols, int ld) {
  constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
  griddep_launch_dependents();
  griddep_wait();
  const int per_row = ld / 8;
  const int64_t n = (a.rows + b.rows) * per_row, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    int64_t row = i / per_row;
    const int col = static_cast<int>(i - row * per_row) * 8;
    const bool second = row >= a.rows;
    const Pack<T> &o = second ? b : a;
    if (second) row -= a.rows;
    VecOf<__nv_bfloat16, 8> out[kPlanes];
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = col + e < cols ? to_f(o.src[row * cols + col + e]) : 0.0f;
    planes_of<kPlanes>(v, out);
#pragma unroll
    for (int q = 0; q < kPlanes; ++q)
      *reinterpret_cast<VecOf<__nv_bfloat16, 8> *>(o.dst + (q * o.rows + row) * ld + col) = out[q];
  }
}

// dz = dy act'(z) as a product's operand (planes and row length as above; null where dy itself
// serves) and its column sums over `block_rows` rows, part[row block][N] (db itself where there is
// one block).  bf16 has one plane: the rounding leaves 0.0023 of the gradients' size in error where
// their own rounding is 0.0017, and a second plane would double the products.  A CTA takes 64
// columns: 8 threads of 8 columns x 32 rows at a time.
constexpr int kDbCols = 64;
template <typename T, int kAct>
__global__ void __launch_bounds__(256)
    proj_dz_kernel(const T *dy, const T *z, __nv_bfloat16 *dz, float *part, int64_t M, int N,
                   int ld, int vec, int block_rows) {
  constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1, V = 16 / static_cast<int>(sizeof(T));
  __shared__ float sums[32][kDbCols + 1];
  griddep_launch_dependents();
  griddep_wait();
  const int c8 = threadIdx.x % 8, rr = threadIdx.x / 8;
  const int col = blockIdx.x * kDbCols + c8 * 8;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * block_rows;
  float sum[8] = {};
  for (int r = rr; r < block_rows; r += 32) {
    const int64_t row = row0 + r;
    if (row >= M || col >= ld) break;
    float d[8];
    const int64_t at = row * N + col;
    if (vec && col + 8 <= N) {
#pragma unroll
      for (int i0 = 0; i0 < 8; i0 += V) {
        const VecOf<T, V> g = *reinterpret_cast<const VecOf<T, V> *>(dy + at + i0);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i0 + i] = to_f(g.e[i]);
        if constexpr (kAct != kNone) {
          const VecOf<T, V> zv = *reinterpret_cast<const VecOf<T, V> *>(z + at + i0);
#pragma unroll
          for (int i = 0; i < V; ++i) d[i0 + i] *= act_slope<T, kAct>(to_f(zv.e[i]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = col + i < N ? to_f(dy[at + i]) : 0.0f;
        if (kAct != kNone && col + i < N) d[i] *= act_slope<T, kAct>(to_f(z[at + i]));
      }
    }
    if (dz) {
      VecOf<__nv_bfloat16, 8> o[kPlanes];
      planes_of<kPlanes>(d, o);
#pragma unroll
      for (int q = 0; q < kPlanes; ++q)
        *reinterpret_cast<VecOf<__nv_bfloat16, 8> *>(dz + (q * M + row) * ld + col) = o[q];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += d[e];
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[rr][c8 * 8 + e] = sum[e];
  __syncthreads();
  if (threadIdx.x < kDbCols && blockIdx.x * kDbCols + threadIdx.x < N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sums[i][threadIdx.x];
    part[static_cast<int64_t>(blockIdx.y) * N + blockIdx.x * kDbCols + threadIdx.x] = s;
  }
}

// db[n]: the sum of the row blocks' sums, in order within each of 8 threads, then over them.
__global__ void __launch_bounds__(256)
    proj_db_kernel(const float *part, float *db, int blocks, int N) {
  __shared__ float sums[8][33];
  griddep_launch_dependents();
  griddep_wait();
  const int c = threadIdx.x % 32, r = threadIdx.x / 32, col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < N)
    for (int b = r; b < blocks; b += 8) s += part[static_cast<int64_t>(b) * N + col];
  sums[r][c] = s;
  __syncthreads();
  if (r == 0 && col < N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += sums[i][c];
    db[col] = t;
  }
}

}  // namespace proj
}  // namespace hyena
