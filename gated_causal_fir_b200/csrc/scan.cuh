// scan.cuh -- the gated linear recurrence along time and its gradients (sm_100a).
//
//     x_t = k_t v_t,   s_t = a_t s_{t-1} + x_t,   y_t = q_t s_t,   a_t = exp(g_t)
//
// for every channel of [B, L, D], with one log decay g per token and group of d_g channels.  A
// run of rows maps the state before it to the state after it by s -> A s + S (A the product of
// its decays, S its result from a zero state), and runs compose: (A2, S2) after (A1, S1) is
// (A2 A1, A2 S1 + S2).  The gradients obey the same recurrence backwards in time,
//
//     u_t = q_t dy_t + w_{t+1},   w_t = a_t u_t      (u = dLoss/ds_t, w what reaches s_{t-1})
//     dq = dy s,   dk = u v,   dv = u k,   dg = sum over the group of w_t s_{t-1}.
//
// Split: a CTA owns 32 channels of one sequence and walks its rows in tiles of 16 R.  (A row of
// 32 channels is 64 bytes in bf16.  At D = 4096 that gives 128 CTAs; a wider piece would leave most
// of the 148 SMs without work.)  Where a problem has too few such columns for the device, its time
// axis is shared as well: by a cluster of CTAs that take neighbouring tiles and send each other
// their (A, S) through distributed shared memory, or by cuts, whose (A, S) a first pass over k, v
// and g finds and every CTA of the second pass joins.  Either way the sums have one order and the
// result is the same in every run.
//
// Within a CTA: one warp streams the tiles in with TMA through a ring of shared-memory stages;
// eight warps compute.  Half a warp (16 lanes of 2 channels) owns a segment of R consecutive
// rows: it takes the segment into registers, frees the stage, forms the segment's (A, S) and joins
// it with the other half's, and after one barrier every lane joins the 8 warps' of its channels in
// order, which gives each its own start and all of them the next tile's.  R is odd for bf16: the two halves of a
// warp then read rows an odd number of 64-byte rows apart, from different banks.
//
// All arithmetic is fp32; q, k, v, g, dy are read once, y, dq, dk, dv, dg rounded once.
// Bound: HBM bandwidth (4 flops per 8 bytes in bf16).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "ptx.cuh"

namespace hyena {
namespace scan {

constexpr int kCh = 32;               // channels of a CTA
constexpr int kSegs = 16;             // segments of a tile: 8 warps x 2 halves
constexpr int kComputeThreads = 256;
constexpr int kHelperWarps = 4;       // warp 0 of them issues TMA, 1..3 form decays (12 warps in
                                      // all: 3 per scheduler start with 168 registers a thread)
constexpr int kThreads = kComputeThreads + 32 * kHelperWarps;
constexpr int kMaxStages = 8;
constexpr unsigned int kTimeout = 1u; // HYENA_DEVICE_TIMEOUT

// How a tile's inputs reach shared memory: the streams by TMA, or where their rows are no multiple
// of 16 bytes by asynchronous 8- or 4-byte copies (single elements where not even those are
// aligned).  One decay per channel: g is a stream like k and v and the compute warps take its exp.
// One per group: the helper warps do, except for groups of few channels (kTmaRaw), whose many exps
// are quicker where they are used (choose_feed on the host has the measurements).
enum Feed { kTmaChannel = 0, kTmaGroup = 1, kCopyChannel = 2, kCopyGroup = 3, kTmaRaw = 4 };
__host__ __device__ constexpr bool by_tma(int feed) {
  return feed == kTmaChannel || feed == kTmaGroup || feed == kTmaRaw;
}
__host__ __device__ constexpr bool per_channel(int feed) {
  return feed == kTmaChannel || feed == kCopyChannel;
}
// Groups' rows of g: a tile by TMA; by 4-byte copies where their rows are no multiple of 16 bytes;
// or element loads (odd numbers of groups in bf16).
enum GroupFeed { kGroupsElement = 0, kGroupsTma = 1, kGroupsCopy = 2 };

// An element type with R, the rows of a segment (a tile has 16 R).  The joining of segments costs
// the same per tile whatever R is, so it takes as many as registers and the ring allow.  B=1 L=8192
// D=4096 bf16, forward and backward in us, d_g = 64 | d_g = 1, and L=65536 D=500 d_g=1:
//     R =  9   55, 109 | 60, 103 | 120, 224
//     R = 11   49, 107 | 57,  98 | 115, 214
//     R = 13   49, 101 | 64,  97 | 128, 279   (rings of two or three stages where g is a stream)
template <typename E, int kRows>
struct Cfg {
  using T = E;
  static constexpr int R = kRows;
};
using Bf16 = Cfg<__nv_bfloat16, 11>;
using F32 = Cfg<float, 7>;

template <typename C>
__host__ __device__ constexpr int tile_rows() { return kSegs * C::R; }
template <typename C>
__host__ __device__ constexpr int stream_bytes() {
  return tile_rows<C>() * kCh * static_cast<int>(sizeof(typename C::T));
}

// fp32 decays of a tile's rows and groups, rounded up to keep what follows them aligned.
template <typename C>
__host__ __device__ constexpr int decay_bytes(int pieces) {
  return (tile_rows<C>() * pieces * 4 + 127) / 128 * 128;
}

struct Params {
  const void *q, *k, *v, *g, *dy;
  const float *s0;                  // [B, D] or null
  const float *ds_out;              // [B, D] or null (backward)
  float *s_out;                     // [B, D] or null: the last state
  float *ds0;                       // [B, D] or null (backward)
  float *ckpt;                      // [B, n_tiles, D]: the state before each tile (fwd writes,
                                    // bwd reads), or null
  float2 *agg;                      // [B, splits, D]: (A, S) of each time cut
  void *y, *dq, *dk, *dv, *dg;
  float *dg_part;                   // [B, L, n_cb] or [B, L, D] partial sums of dg
  unsigned int *status;
  int B, L, D, d_g, G;
  int n_cb, n_tiles, splits, tiles_per_split;
  int unit_split0, unit_splits;     // the cuts this launch works on
  int n_units;                      // B x unit_splits x n_cb
  int cluster;                      // CTAs that share a unit's tiles (kCl)
  int pieces, piece_bits;           // groups a block of 32 channels touches at most; and the
                                    // least power of two that holds them
  int g_feed;                       // how the groups' rows of g arrive (GroupFeed)
  int copy_bits;                    // least power of two of copies per row of theirs
  int g_align, g_box;               // their tile starts at a multiple of g_align groups, g_box wide
  int copy;                         // bytes per asynchronous copy: 8, 4, or 0 for element loads
  int pair_out;                     // rows and bases allow stores of two channels
  int stages, stage_bytes;
  int dg_mode;                      // 0: dg itself, 1: one partial per block, 2: per channel
  uint64_t wait_ns;                 // limit of a cluster's waits (2 s but in tests)
  int fault;                        // test hook: 1: rank 0 of a cluster withholds its first (A, S)
};

// ---------------------------------------------------------------------------- two channels
// A lane's two channels as one packed pair of fp32 (fma.f32x2 takes both in one instruction).
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// The two channels of a row as they lie in shared memory.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  __device__ static F2 f(Raw r) {
    return pack(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  __device__ static void store(__nv_bfloat16 *p, F2 v) {
    const float2 x = unpack(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
    *reinterpret_cast<__nv_bfloat162 *>(p) = b;
  }
};
template <> struct Pair<float> {
  using Raw = F2;
  __device__ static F2 f(Raw r) { return r; }
  __device__ static void store(float *p, F2 x) { *reinterpret_cast<F2 *>(p) = x; }
};
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store_one(float *p, float x) { *p = x; }
__device__ __forceinline__ float load_one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_one(const float *p) { return *p; }

// exp(g), accurately: a state sums hundreds of products of decays, and the faster 2^x (with its
// 2^-22) left the states three times as far off, for 4 us of 62 (B=1 L=8192 D=4096 d_g=1).
__device__ __forceinline__ float decay(float g) { return expf(g); }

__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory");
}

// ---------------------------------------------------------------------------- a CTA's ring
constexpr int kStageAlign = 128;  // of a TMA destination
__device__ __forceinline__ uint8_t *align_stage(uint8_t *dynamic) {
  return dynamic + (kStageAlign - smem_u32(dynamic) % kStageAlign) % kStageAlign;
}

struct Ring {
  uint64_t full[kMaxStages], empty[kMaxStages], raw[kMaxStages];  // raw: g's tile has landed
  int abort;
};

// The work unit `u`: channel block fastest, so that neighbouring CTAs read neighbouring pieces of
// the same rows.
struct Unit {
  int b, cb, split, tile0, tile1;
  __device__ Unit(const Params &p, int u) {
    cb = u % p.n_cb;
    const int r = u / p.n_cb;
    split = p.unit_split0 + r % p.unit_splits;
    b = r / p.unit_splits;
    tile0 = split * p.tiles_per_split;
    tile1 = min(tile0 + p.tiles_per_split, p.n_tiles);
  }
};

// The tiles of a unit that this CTA takes: `first`, then every step-th up to (kReverse: down to)
// the unit's bound.  kCl: every cluster-th one, in rounds; the last (kReverse: first) round may lie
// past the unit's tiles for it.
template <bool kCl, bool kReverse>
struct Walk {
  int first, step, end;
  __device__ Walk(const Params &p, const Unit &u, int rank) {
    const int size = kCl ? p.cluster : 1;
    const int rounds = (u.tile1 - u.tile0 + size - 1) / size;
    first = u.tile0 + (kReverse ? (rounds - 1) * size : 0) + (kCl ? rank : 0);
    step = kReverse ? -size : size;
    end = kReverse ? u.tile0 : u.tile0 + rounds * size;
  }
  __device__ bool more(int tile) const { return kReverse ? tile >= end : tile < end; }
};

// The CTA's rank in its cluster.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// What the CTAs of a cluster tell each other in a round: the (A, S) of the tile that each took.
struct Exchange {
  ulonglong2 of[2][8][kCh / 2];
  uint64_t all[2];  // the round's bytes from every CTA
};
constexpr int kMaxCluster = 8;

// Sends this tile's (A, S) (one warp; lane l and 16 + l hold the same) to every CTA of the cluster:
// stores that count their bytes on the receiver's barrier, one way.  A CTA that has given up sends
// no more: the phase that it gave up on is open, and may not be armed a second time.
__device__ __forceinline__ void send(Exchange &x, int round, int rank, int size, F2 A, F2 S,
                                     int fault) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) mbar_arrive_expect_tx(&x.all[round & 1], size * (kCh / 2) * 16);
  const uint32_t slot = smem_u32(&x.of[round & 1][rank][lane % 16]);
  const uint32_t bar = smem_u32(&x.all[round & 1]);
  if (fault == 1 && round == 0 && rank == 0) return;
  for (int to = lane / 16; to < size; to += 2)
    asm volatile(
        "{\n\t.reg .u32 a, b;\n\tmapa.shared::cluster.u32 a, %0, %2;\n\t"
        "mapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [a], {%3, %4}, [b];\n\t}" ::"r"(
            slot),
        "r"(bar), "r"(to), "l"(A), "l"(S)
        : "memory");
}
// Waits until every CTA's word of this round is here.
__device__ __forceinline__ bool received(Exchange &x, int round, Ring &ring, const Params &p) {
  return mbar_wait(&x.all[round & 1], (round >> 1) & 1, &ring.abort, p.status, kTimeout, p.wait_ns);
}

// One decay per row and group of the block by the warps [0, warps): lanes take groups first, in a
// power of two of columns (p.piece_bits), so that no index is divided; g_at(row, group) is the log
// decay, and 0 past the end, where rows leave the state as it is.
template <typename C, int kBatch, typename F>  // kBatch: loads in flight per thread
__device__ __forceinline__ void form_batches(const Params &p, float *as, int warp, int warps,
                                             F &&g_at) {
  const int lane = threadIdx.x % 32, per = 32 >> p.piece_bits;  // rows a warp takes at a time
  const int gi = lane & ((1 << p.piece_bits) - 1);
  if (gi >= p.pieces) return;
  const int step = warps * per;
  for (int row = warp * per + (lane >> p.piece_bits); row < tile_rows<C>(); row += kBatch * step) {
    float v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      v[i] = row + i * step < tile_rows<C>() ? g_at(row + i * step, gi) : 0.0f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (row + i * step < tile_rows<C>()) as[(row + i * step) * p.pieces + gi] = decay(v[i]);
  }
}
template <typename C, typename F>
__device__ __forceinline__ void form_decays(const Params &p, float *as, int warp, int warps,
                                            F &&g_at) {
  if (p.piece_bits <= 1)
    form_batches<C, 4>(p, as, warp, warps, g_at);
  else
    form_batches<C, 24>(p, as, warp, warps, g_at);
}

// From global memory.
template <typename C>
__device__ __forceinline__ void fill_decays(const Params &p, float *as, int b, int c0, int t0,
                                            int warp, int warps) {
  using T = typename C::T;
  const int g0 = c0 / p.d_g, rows = p.L - t0, groups = p.G - g0;
  const T *g = static_cast<const T *>(p.g) + (static_cast<int64_t>(b) * p.L + t0) * p.G + g0;
  form_decays<C>(p, as, warp, warps, [&](int row, int gi) {
    return row < rows && gi < groups ? load_one(g + static_cast<int64_t>(row) * p.G + gi) : 0.0f;
  });
}

// From the tile of g's rows in shared memory (zeros past the end).
template <typename C>
__device__ __forceinline__ void convert_decays(const Params &p, float *as,
                                               const typename C::T *g, int first, int warp,
                                               int warps) {
  form_decays<C>(p, as, warp, warps,
                 [&](int row, int gi) { return load_one(g + row * p.g_box + first + gi); });
}

// One stream's tile by the helper threads' asynchronous copies; zero outside the tensor, as TMA
// fills.
template <typename C, int kBytes>
__device__ __forceinline__ void copy_tile(const Params &p, typename C::T *dst, const void *src,
                                          int b, int c0, int t0, int thread) {
  using T = typename C::T;
  constexpr int E = kBytes / static_cast<int>(sizeof(T)), N = kCh / E;  // elements; copies per row
  constexpr int kStep = 32 * kHelperWarps / N;                          // rows apart
  static_assert(E >= 1 && 32 * kHelperWarps % N == 0, "copies of a row");
  constexpr int kCopies = tile_rows<C>() / kStep;
  static_assert(kCopies * kStep == tile_rows<C>(), "copies of a column");
  const int c = c0 + thread % N * E, row0 = thread / N;
  const bool inside = c < p.D;
  const uint8_t *s = static_cast<const uint8_t *>(src);
  if (inside)
    s += ((static_cast<int64_t>(b) * p.L + t0 + row0) * p.D + c) * static_cast<int64_t>(sizeof(T));
  const int64_t step = inside ? static_cast<int64_t>(kStep) * p.D * static_cast<int64_t>(sizeof(T)) : 0;
  const uint32_t d = smem_u32(dst + row0 * kCh + thread % N * E);
  const int rows = inside ? p.L - t0 - row0 : 0;  // rows of this thread's, and between, to read
  if (p.L - t0 >= tile_rows<C>()) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i, s += step)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                       d + i * kStep * kCh * static_cast<int>(sizeof(T))),
                   "l"(s), "n"(kBytes), "r"(inside ? kBytes : 0)
                   : "memory");
  } else {
#pragma unroll 1
    for (int i = 0; i < kCopies; ++i) {
      const bool live = i * kStep < rows;
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                       d + i * kStep * kCh * static_cast<int>(sizeof(T))),
                   "l"(live ? s + i * step : static_cast<const uint8_t *>(src)), "n"(kBytes),
                   "r"(live ? kBytes : 0)
                   : "memory");
    }
  }
}

template <typename C>
__device__ __forceinline__ void load_elements(const Params &p, typename C::T *dst,
                                              const void *src, int b, int c0, int t0, int thread) {
  using T = typename C::T;
  const T *s = static_cast<const T *>(src) + static_cast<int64_t>(b) * p.L * p.D;
  for (int e = thread; e < tile_rows<C>() * kCh; e += 32 * kHelperWarps) {
    const int t = t0 + e / kCh, c = c0 + e % kCh;
    dst[e] = t < p.L && c < p.D ? s[static_cast<int64_t>(t) * p.D + c] : T(0.0f);
  }
}

// The tile of the groups' rows of g by the warps [0, warps): 4-byte copies, or element loads; zeros
// past the end.
template <typename C>
__device__ __forceinline__ void groups_tile(const Params &p, typename C::T *dst, int b, int c0,
                                            int t0, int warp, int warps) {
  using T = typename C::T;
  constexpr int E = 4 / static_cast<int>(sizeof(T));  // groups per copy
  const int lane = threadIdx.x % 32, x = c0 / p.d_g / p.g_align * p.g_align;
  const T *g = static_cast<const T *>(p.g) + (static_cast<int64_t>(b) * p.L + t0) * p.G + x;
  const int rows = p.L - t0;
  if (p.g_feed == kGroupsCopy) {
    const int n = p.g_box / E, bits = min(p.copy_bits, 5), per = warps * (32 >> bits);
    for (int col = lane & ((1 << bits) - 1); col < n; col += 32) {
      const bool inside = x + col * E < p.G;
      int row = warp * (32 >> bits) + (lane >> bits);
      const T *from = g + static_cast<int64_t>(row) * p.G + col * E;
      uint32_t to = smem_u32(dst + row * p.g_box + col * E);
      const int64_t step = static_cast<int64_t>(per) * p.G;
      const uint32_t to_step = per * p.g_box * static_cast<uint32_t>(sizeof(T));
#pragma unroll 4
      for (; row < tile_rows<C>(); row += per, from += step, to += to_step) {
        const bool live = inside && row < rows;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to),
                     "l"(live ? from : static_cast<const T *>(p.g)), "r"(live ? 4 : 0)
                     : "memory");
      }
    }
  } else {
    constexpr int kBatch = 16;  // loads in flight per thread
    for (int e0 = warp * 32 + lane; e0 < tile_rows<C>() * p.g_box; e0 += kBatch * warps * 32) {
      T v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = (e0 + i * warps * 32) / p.g_box, gi = e0 + i * warps * 32 - row * p.g_box;
        v[i] = row < tile_rows<C>() && row < rows && x + gi < p.G
                   ? g[static_cast<int64_t>(row) * p.G + gi]
                   : T(0.0f);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (e0 + i * warps * 32 < tile_rows<C>() * p.g_box) dst[e0 + i * warps * 32] = v[i];
    }
  }
}

// Arrives on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Which arrivals a helper thread of a copying feed makes on a tile's barrier: one when its copies
// have landed, one (a release) for what it stored itself.  Groups' rows that TMA could take are
// stored by elements here too, as groups_tile does with all that it does not copy.
template <int kFeed>
__device__ __forceinline__ bool copy_arrivals(const Params &p) {
  return p.copy || (!per_channel(kFeed) && p.g_feed == kGroupsCopy);
}
template <int kFeed>
__device__ __forceinline__ bool store_arrivals(const Params &p) {
  return !p.copy || (!per_channel(kFeed) && p.g_feed != kGroupsCopy);
}

// The helper warps: NS streams of every tile of the CTA's units into the ring, in the order the
// compute warps take them (kReverse: last tile first).
template <typename C, int kFeed, bool kReverse, int NS, bool kCl>
__device__ __forceinline__ void feed(const Params &p, Ring &ring, uint8_t *stages,
                                     const CUtensorMap *const (&maps)[5],
                                     const void *const (&ptrs)[5]) {
  using T = typename C::T;
  const int warp = threadIdx.x / 32 - kComputeThreads / 32, lane = threadIdx.x % 32;
  constexpr int kStreams = NS + (per_channel(kFeed) ? 1 : 0);
  constexpr int kBytes = stream_bytes<C>();
  const int th = threadIdx.x - kComputeThreads;
  // the groups' warps in a TMA feed: where their rows are copied, warp 1 copies and the rest of the
  // helpers form decays; all of them copy where the compute warps take the exps
  const bool copies = p.g_feed == kGroupsCopy;
  const int converters = kFeed == kTmaGroup ? kHelperWarps - (copies ? 2 : 1) : 0;
  const int copiers = copies ? kHelperWarps - 1 - converters : 0;
  const bool converter = warp >= kHelperWarps - converters;
  if (by_tma(kFeed) && warp == 0 && lane != 0) return;
  if (kFeed == kTmaChannel && warp != 0) return;
  if (kFeed == kTmaRaw && warp != 0 && !copies) return;
  int it = 0, last = 0;
  const int size = kCl ? p.cluster : 1, rank = kCl ? cluster_rank() : 0;
  for (int u = blockIdx.x / size; u < p.n_units; u += gridDim.x / size) {
    const Unit un(p, u);
    const Walk<kCl, kReverse> walk(p, un, rank);
    const int c0 = un.cb * kCh;
    for (int tile = walk.first; walk.more(tile); tile += walk.step) {
      if (kCl && tile >= un.tile1) continue;
      const int t0 = tile * tile_rows<C>();
      const int st = it % p.stages, round = it / p.stages;
      uint8_t *buf = stages + st * p.stage_bytes;
      float *as = reinterpret_cast<float *>(buf + NS * kBytes);  // decays (kTmaGroup)
      T *graw = reinterpret_cast<T *>(
          buf + NS * kBytes + (kFeed == kTmaGroup ? decay_bytes<C>(p.pieces) : 0));
      uint64_t *graw_full = kFeed == kTmaGroup ? &ring.raw[st] : &ring.full[st];
      if (round > 0 && !mbar_wait(&ring.empty[st], (round - 1) & 1, &ring.abort, p.status, kTimeout))
        goto out;
      if (by_tma(kFeed) && warp == 0) {
        int bytes = kStreams * kBytes;
        if (!per_channel(kFeed) && p.g_feed == kGroupsTma) {
          const int graw_bytes = tile_rows<C>() * p.g_box * static_cast<int>(sizeof(T));
          if (kFeed == kTmaGroup)
            mbar_arrive_expect_tx(graw_full, graw_bytes);
          else
            bytes += graw_bytes;
        }
        mbar_arrive_expect_tx(&ring.full[st], bytes);
        if (!per_channel(kFeed) && p.g_feed == kGroupsTma)
          tma_load_3d(graw, maps[4], graw_full, c0 / p.d_g / p.g_align * p.g_align, t0, un.b);
#pragma unroll
        for (int s = 0; s < kStreams; ++s)
          tma_load_3d(buf + s * kBytes, maps[s], &ring.full[st], c0, t0, un.b);
        last = it + 1;
      } else if (by_tma(kFeed) && !per_channel(kFeed) && warp <= copiers) {
        groups_tile<C>(p, graw, un.b, c0, t0, warp - 1, copiers);
        arrive_after_copies(graw_full);
      } else if (kFeed == kTmaGroup && converter) {
        const int w = warp - (kHelperWarps - converters);
        if (p.g_feed == kGroupsElement) {
          fill_decays<C>(p, as, un.b, c0, t0, w, converters);
        } else {
          if (!mbar_wait(&ring.raw[st], round & 1, &ring.abort, p.status, kTimeout)) goto out;
          convert_decays<C>(p, as, graw, c0 / p.d_g % p.g_align, w, converters);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.full[st]);
      } else if (!by_tma(kFeed)) {
#pragma unroll
        for (int s = 0; s < kStreams; ++s) {
          T *dst = reinterpret_cast<T *>(buf + s * kBytes);
          if (p.copy == 8)
            copy_tile<C, 8>(p, dst, ptrs[s], un.b, c0, t0, th);
          else if (p.copy == 4)
            copy_tile<C, 4>(p, dst, ptrs[s], un.b, c0, t0, th);
          else
            load_elements<C>(p, dst, ptrs[s], un.b, c0, t0, th);
        }
        if (!per_channel(kFeed)) groups_tile<C>(p, graw, un.b, c0, t0, warp, kHelperWarps);
        // one arrival for the copies, and one for what the thread stored itself
        if (copy_arrivals<kFeed>(p)) arrive_after_copies(&ring.full[st]);
        if (store_arrivals<kFeed>(p)) mbar_arrive(&ring.full[st]);
      }
      ++it;
    }
  }
out:
  // no copy may be in flight when the CTA ends, whatever happened to the readers
  if (by_tma(kFeed) && warp == 0) {
    for (int j = max(0, last - p.stages); j < last; ++j) {
      int no_abort = 0;
      if (kFeed == kTmaGroup && p.g_feed == kGroupsTma)
        mbar_wait(&ring.raw[j % p.stages], (j / p.stages) & 1, &no_abort, p.status, kTimeout);
      mbar_wait(&ring.full[j % p.stages], (j / p.stages) & 1, &no_abort, p.status, kTimeout);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int kFeed>
__device__ __forceinline__ void ring_init(const Params &p, Ring &ring) {
  if (threadIdx.x == 0) {
    const bool copies = p.g_feed == kGroupsCopy;
    int arrivals = 1;  // the TMA warp
    if (kFeed == kTmaGroup) arrivals += kHelperWarps - (copies ? 2 : 1);
    if (kFeed == kTmaRaw && copies) arrivals += 32 * (kHelperWarps - 1);
    if (!by_tma(kFeed))
      arrivals = 32 * kHelperWarps * (copy_arrivals<kFeed>(p) + store_arrivals<kFeed>(p));
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ring.full[i], arrivals);
      mbar_init(&ring.empty[i], kComputeThreads / 32);
      mbar_init(&ring.raw[i], copies ? 32 : 1);
    }
    ring.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
}

// A lane's decays in the rows of its segment.
template <typename C, int kFeed, bool kChannel = per_channel(kFeed)> struct Decays;
template <typename C, int kFeed>
struct Decays<C, kFeed, true> {  // from the lane's pairs of g
  using T = typename C::T;
  using Held = F2;
  const uint8_t *at;
  __device__ Decays(const Params &, const uint8_t *tile, int seg, int l, int)
      : at(tile + (seg * C::R * kCh + 2 * l) * static_cast<int>(sizeof(T))) {}
  __device__ Held load(int r) const {
    const float2 g = unpack(Pair<T>::f(*reinterpret_cast<const typename Pair<T>::Raw *>(
        at + r * kCh * static_cast<int>(sizeof(T)))));
    return pack(decay(g.x), decay(g.y));
  }
  __device__ static F2 pair(Held a) { return a; }
};
template <typename C>
struct Decays<C, kTmaGroup, false> {  // d_g is even: the two channels share one
  using Held = float;
  const float *at;
  int step;
  __device__ Decays(const Params &p, const uint8_t *tile, int seg, int l, int c0) {
    const int c = min(c0 + 2 * l, p.D - 1);
    at = reinterpret_cast<const float *>(tile) + seg * C::R * p.pieces + c / p.d_g -
         c0 / p.d_g;
    step = p.pieces;
  }
  __device__ Held load(int r) const { return at[r * step]; }
  __device__ static F2 pair(Held a) { return pack(a, a); }
};
template <typename C>
struct Decays<C, kTmaRaw, false> {  // the same, from the tile of g's rows
  using T = typename C::T;
  using Held = float;
  const T *at;
  int step;
  __device__ Decays(const Params &p, const uint8_t *tile, int seg, int l, int c0) {
    const int c = min(c0 + 2 * l, p.D - 1), g0 = c0 / p.d_g;
    at = reinterpret_cast<const T *>(tile) + seg * C::R * p.g_box + g0 % p.g_align + c / p.d_g -
         g0;
    step = p.g_box;
  }
  __device__ Held load(int r) const { return decay(load_one(at + r * step)); }
  __device__ static F2 pair(Held a) { return pack(a, a); }
};
template <typename C>
struct Decays<C, kCopyGroup, false> {  // any d_g
  using T = typename C::T;
  using Held = F2;
  const T *at;
  int step, second;
  __device__ Decays(const Params &p, const uint8_t *tile, int seg, int l, int c0) {
    const int g0 = c0 / p.d_g, i0 = min(c0 + 2 * l, p.D - 1) / p.d_g - g0;
    at = reinterpret_cast<const T *>(tile) + seg * C::R * p.g_box + g0 % p.g_align + i0;
    second = min(c0 + 2 * l + 1, p.D - 1) / p.d_g - g0 - i0;
    step = p.g_box;
  }
  __device__ Held load(int r) const {
    const float a = decay(load_one(at + r * step));
    return pack(a, second ? decay(load_one(at + r * step + second)) : a);
  }
  __device__ static F2 pair(Held a) { return a; }
};

// A lane's two channels in consecutive rows of a [B, L, D] tensor, from (b, t0) on; rows past the
// end and channels past D are not written (live: rows to write; hi: whether the second is inside).
template <typename T, int kFeed>
struct Out {
  T *at;
  uint32_t stride;  // bytes per row; D is below 2^28
  int live;
  bool hi, pairs;
  __device__ Out(void *base, const Params &p, int b, int t0, int c, bool dead) {
    at = static_cast<T *>(base) + (static_cast<int64_t>(b) * p.L + t0) * p.D + c;
    stride = static_cast<uint32_t>(p.D) * static_cast<uint32_t>(sizeof(T));
    live = dead || c >= p.D ? 0 : p.L - t0;
    hi = c + 1 < p.D;
    pairs = by_tma(kFeed) || p.pair_out;
  }
  // kWhole: all rows up to r are inside (live > r)
  template <bool kWhole = false>
  __device__ void put(int r, F2 x) const {
    if (!kWhole && r >= live) return;
    T *to = reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(at) +
                                  static_cast<uint64_t>(stride) * static_cast<uint32_t>(r));
    if (pairs) {  // D is even: a pair is inside or outside
      Pair<T>::store(to, x);
    } else {
      const float2 v = unpack(x);
      store_one(to, v.x);
      if (hi) store_one(to + 1, v.y);
    }
  }
};

__device__ __forceinline__ F2 get_state(const float *s, int64_t row, int c, int D) {
  if (!s) return 0;
  s += row * D;
  return pack(c < D ? s[c] : 0.f, c + 1 < D ? s[c + 1] : 0.f);
}
__device__ __forceinline__ void put_state(float *s, int64_t row, int c, int D, F2 v) {
  const float2 x = unpack(v);
  s += row * D;
  if (c < D) s[c] = x.x;
  if (c + 1 < D) s[c + 1] = x.y;
}
// s after the cut with (A, S) in agg[c], agg[c + 1]
__device__ __forceinline__ F2 through_cut(const float2 *agg, int c, int D, F2 v) {
  float2 s = unpack(v);
  if (c < D) s.x = fmaf(agg[c].x, s.x, agg[c].y);
  if (c + 1 < D) s.y = fmaf(agg[c + 1].x, s.y, agg[c + 1].y);
  return pack(s.x, s.y);
}
__device__ __forceinline__ void put_cut(float2 *agg, int c, int D, F2 a, F2 v) {
  const float2 A = unpack(a), S = unpack(v);
  if (c < D) agg[c] = make_float2(A.x, S.x);
  if (c + 1 < D) agg[c + 1] = make_float2(A.y, S.y);
}

// Reads every loaded word in an instruction that cannot be left out, so that the warp waits until
// the loads have returned: what is only used after its stage has been handed back could otherwise
// still be in flight when the next tile's copy lands there.  (B=1 L=8192 D=4096 bf16 d_g=64: 47.1 us
// without, 47.7 with it.)
template <typename Raw, int R>
__device__ __forceinline__ void consume(const Raw (&v)[R]) {
  Raw any = v[0];
#pragma unroll
  for (int r = 1; r < R; ++r) any |= v[r];
  const uint32_t word = static_cast<uint32_t>(any) | static_cast<uint32_t>(static_cast<uint64_t>(any) >> 32);
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %0, 0xfffffffe;\n\t@p nanosleep.u32 0;\n\t}" ::"r"(
      word));
}

constexpr F2 kOnes = 0x3f8000003f800000ull;
constexpr int kWarps = kComputeThreads / 32;

__device__ __forceinline__ F2 from_other_half(F2 x) { return __shfl_xor_sync(0xffffffffu, x, 16); }

// The cluster's barriers exist before a peer arrives on them, and a CTA stays until the last has.
__device__ __forceinline__ void exchange_init(Exchange &x) {
  if (threadIdx.x == 0) {
    mbar_init(&x.all[0], 1);
    mbar_init(&x.all[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  cluster_sync();
}
__device__ __forceinline__ void exchange_end(bool gave_up) {
  __syncwarp();
  cluster_sync();
  // What peers sent in rounds that this CTA gave up on lands within a few microseconds; nobody
  // waits for those bytes, so the CTA stays while they arrive.
  if (gave_up) {
    const uint64_t t0 = global_timer_ns();
    for (int i = 0; i < 10000 && global_timer_ns() - t0 < 200000; ++i) __nanosleep(1000);
  }
}

// ---------------------------------------------------------------------------- forward
// kOut: y and the last state (streams k, v, q); otherwise only states: checkpoints, or the (A, S)
// of the unit's time cut from a zero state (streams k, v).
template <typename C, int kFeed, bool kOut, bool kCl>
__global__ void __launch_bounds__(kThreads, 1)
    scan_fwd_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                    const Params p) {
  extern __shared__ uint8_t dynamic[];
  uint8_t *stages = align_stage(dynamic);
  __shared__ Ring ring;
  __shared__ ulonglong2 joint[2][kWarps][kCh / 2];  // (A, S) of a warp's rows
  using T = typename C::T;
  constexpr int R = C::R, NS = kOut ? 3 : 2, kBytes = stream_bytes<C>();
  using Raw = typename Pair<T>::Raw;
  using Dec = Decays<C, kFeed>;
  __shared__ Exchange xch;
  ring_init<kFeed>(p, ring);
  if (kCl) exchange_init(xch);
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x >= kComputeThreads) {
    const CUtensorMap *const maps[5] = {&mk, &mv, kOut ? &mq : &mg, &mg, &mg};
    const void *const ptrs[5] = {p.k, p.v, kOut ? p.q : p.g, p.g, nullptr};
    feed<C, kFeed, false, NS, kCl>(p, ring, stages, maps, ptrs);
    if (kCl) exchange_end(false);
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % 16;
  const int seg = threadIdx.x / 16;
  const bool second = lane >= 16;
  const int size = kCl ? p.cluster : 1, rank = kCl ? cluster_rank() : 0;
  bool dead = false;
  int round = 0, empty = 0;  // tiles, and rounds without one
  for (int u = blockIdx.x / size; u < p.n_units; u += gridDim.x / size) {
    const Unit un(p, u);
    const int c0 = un.cb * kCh, c = c0 + 2 * l;
    const bool from_zero = !kOut && !p.ckpt;  // (A, S) of a cut
    float2 *agg = p.agg + static_cast<int64_t>(un.b) * p.splits * p.D;
    F2 carry = 0, whole = kOnes;
    if (!from_zero) {  // the state before the unit: s0 through the cuts before it
      carry = get_state(p.s0, un.b, c, p.D);
      for (int j = 0; j < un.split; ++j)
        carry = through_cut(agg + static_cast<int64_t>(j) * p.D, c, p.D, carry);
    }
    const Walk<kCl, false> walk(p, un, rank);
    for (int tile = walk.first; walk.more(tile); tile += walk.step, ++round) {
      const int buffer = round & 1;
      if (kCl && tile >= un.tile1) {  // an empty round: the state passes unchanged
        compute_barrier();  // nobody here still reads what peers may overwrite after this send
        if (warp == 0 && !dead) send(xch, round, rank, size, kOnes, 0, p.fault);
        if (!received(xch, round, ring, p)) dead = true;
        for (int j = 0; j < size; ++j) {
          const ulonglong2 m = xch.of[buffer][j][l];
          carry = fma2(m.x, carry, m.y);
        }
        ++empty;
        continue;
      }
      const int it = kCl ? round - empty : round, st = it % p.stages;
      const uint8_t *buf = stages + st * p.stage_bytes;
      if (!mbar_wait(&ring.full[st], (it / p.stages) & 1, &ring.abort, p.status, kTimeout))
        dead = true;
      F2 x[R];
      typename Dec::Held a[R];
      Raw qr[R];
      const Dec dec(p, buf + NS * kBytes, seg, l, c0);
      const uint8_t *at = buf + (seg * R * kCh + 2 * l) * static_cast<int>(sizeof(T));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int o = r * kCh * static_cast<int>(sizeof(T));
        x[r] = mul2(Pair<T>::f(*reinterpret_cast<const Raw *>(at + o)),
                    Pair<T>::f(*reinterpret_cast<const Raw *>(at + kBytes + o)));
        if (kOut) qr[r] = *reinterpret_cast<const Raw *>(at + 2 * kBytes + o);
        a[r] = dec.load(r);
      }
      F2 A = Dec::pair(a[0]), S = x[0];
#pragma unroll
      for (int r = 1; r < R; ++r) {
        S = fma2(Dec::pair(a[r]), S, x[r]);
        A = mul2(A, Dec::pair(a[r]));
      }
      // the halves of the warp, joined by the first; the second keeps the first's
      const F2 Ao = from_other_half(A), So = from_other_half(S);
      if (!second) joint[buffer][warp][l] = make_ulonglong2(mul2(Ao, A), fma2(Ao, S, So));
      if (kOut) consume(qr);  // (k, v and the decays went into A and S)
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);  // the segment is in registers
      compute_barrier();
      F2 s = carry;
      if constexpr (kCl) {
        // the tile as a whole and up to this warp; then the tiles of the round, in order
        F2 Ap = kOnes, Sp = 0, At = kOnes, St = 0;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) {
          const ulonglong2 m = joint[buffer][j][l];
          if (j == warp) Ap = At, Sp = St;
          St = fma2(m.x, St, m.y);
          At = mul2(At, m.x);
        }
        if (warp == 0 && !dead) send(xch, round, rank, size, At, St, p.fault);
        if (!received(xch, round, ring, p)) dead = true;
#pragma unroll
        for (int j = 0; j < kMaxCluster; ++j) {
          if (j >= size) break;
          const ulonglong2 m = xch.of[buffer][j][l];
          if (j == rank) s = carry;
          carry = fma2(m.x, carry, m.y);
        }
        if (p.ckpt && seg == 0 && !dead)
          put_state(p.ckpt, static_cast<int64_t>(un.b) * p.n_tiles + tile, c, p.D, s);
        s = fma2(Ap, s, Sp);
      } else {
        if (p.ckpt && seg == 0 && !dead)
          put_state(p.ckpt, static_cast<int64_t>(un.b) * p.n_tiles + tile, c, p.D, carry);
#pragma unroll
        for (int j = 0; j < kWarps; ++j) {
          const ulonglong2 m = joint[buffer][j][l];
          if (j == warp) s = carry;
          carry = fma2(m.x, carry, m.y);
          if (!kOut) whole = mul2(whole, m.x);
        }
      }
      if (kOut) {
        if (second) s = fma2(Ao, s, So);
        const Out<T, kFeed> y(p.y, p, un.b, tile * tile_rows<C>() + seg * R, c, dead);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s = fma2(Dec::pair(a[r]), s, x[r]);
          y.put(r, mul2(Pair<T>::f(qr[r]), s));
        }
      }
    }
    if (seg == 0 && !dead) {
      if (p.s_out && un.tile1 == p.n_tiles && rank == 0) put_state(p.s_out, un.b, c, p.D, carry);
      if (from_zero) put_cut(agg + static_cast<int64_t>(un.split) * p.D, c, p.D, whole, carry);
    }
  }
  if (kCl) exchange_end(dead);
}

// ---------------------------------------------------------------------------- backward
// Sums over 2 kHalf neighbouring lanes of one value per row.  Each exchange halves the rows that a
// lane holds: of n rows the upper lane keeps those from h = ceil(n / 2) on and gives the others; an
// odd row out is summed in both.  row(p) is the row that position p holds after the exchanges
// (11 rows over 16 lanes: 12 exchanges where sums of each row would take 44).
template <int kHalf, int n>
struct GroupSum {
  static constexpr int h = (n + 1) / 2;
  using Next = GroupSum<kHalf / 2, h>;
  static constexpr int kLeft = Next::kLeft;
  __device__ static __forceinline__ void sum(float *w, int l) {
    const bool up = l & kHalf;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const bool pair = i + h < n;
      const float give = pair && !up ? w[pair ? i + h : i] : w[i];
      const float keep = pair && up ? w[pair ? i + h : i] : w[i];
      w[i] = keep + __shfl_xor_sync(0xffffffffu, give, kHalf);
    }
    Next::sum(w, l);
  }
  __device__ static __forceinline__ int row(int p, int l) {
    const int i = Next::row(p, l);
    return (l & kHalf) && i + h < n ? i + h : i;
  }
};
template <int n>
struct GroupSum<0, n> {
  static constexpr int kLeft = n;
  __device__ static __forceinline__ void sum(float *, int) {}
  __device__ static __forceinline__ int row(int p, int) { return p; }
};
// put(row, group of lanes, sum) gets each row's.
template <int kSpan, int R, typename F>
__device__ __forceinline__ void sum_groups(float (&v)[R], int l, F &&put) {
  using S = GroupSum<kSpan / 2, R>;
  S::sum(v, l);
#pragma unroll
  for (int i = 0; i < S::kLeft; ++i) put(S::row(i, l), l / kSpan, v[i]);
}

// The backward holds five values a row where the forward holds three, so its compute warps take
// registers from the helpers: a block starts with 65536 / 384, rounded down to a multiple of 8, a
// thread, and the shares sum to what it starts with.  (Without, R = 9 fitted with a few spills,
// and what is spilled leaves the small L1 beside the ring: 119 us at d_g = 64 instead of 107.)
constexpr int kStartRegs = 168, kHelperRegs = 88, kComputeRegs = 208;
static_assert(kComputeThreads % 128 == 0 && kHelperWarps % 4 == 0, "whole warpgroups");
static_assert(kComputeThreads * kComputeRegs + 32 * kHelperWarps * kHelperRegs <=
                  kThreads * kStartRegs,
              "the block's registers");
template <int n>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}

// kOut: the gradients (streams q, dy, k, v and the checkpoints); otherwise the (A, W) of the
// unit's time cut from w = 0 (streams q, dy).
template <typename C, int kFeed, bool kOut, bool kCl>
__global__ void __launch_bounds__(kThreads, 1)
    scan_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdy,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mg, const Params p) {
  extern __shared__ uint8_t dynamic[];
  uint8_t *stages = align_stage(dynamic);
  __shared__ Ring ring;
  __shared__ ulonglong2 joint[2][kWarps][kCh / 2];  // (A, S) of a warp's rows
  __shared__ F2 joint_w[2][kWarps][kCh / 2];
  using T = typename C::T;
  constexpr int R = C::R, NS = kOut ? 4 : 2, kBytes = stream_bytes<C>();
  using Raw = typename Pair<T>::Raw;
  using Dec = Decays<C, kFeed>;
  __shared__ Exchange xch;
  ring_init<kFeed>(p, ring);
  if (kCl) exchange_init(xch);
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x >= kComputeThreads) {
    if (kOut) registers_down<kHelperRegs>();
    const CUtensorMap *const maps[5] = {&mq, &mdy, kOut ? &mk : &mg, &mv, &mg};
    const void *const ptrs[5] = {p.q, p.dy, kOut ? p.k : p.g, p.v, p.g};
    feed<C, kFeed, true, NS, kCl>(p, ring, stages, maps, ptrs);
    if (kCl) exchange_end(false);
    return;
  }
  if (kOut) registers_up<kComputeRegs>();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, l = lane % 16;
  const int seg = threadIdx.x / 16;
  const bool second = lane >= 16;
  const int size = kCl ? p.cluster : 1, rank = kCl ? cluster_rank() : 0;
  bool dead = false;
  int round = 0, empty = 0;  // tiles, and rounds without one
  for (int u = blockIdx.x / size; u < p.n_units; u += gridDim.x / size) {
    const Unit un(p, u);
    const int c0 = un.cb * kCh, c = c0 + 2 * l;
    float2 *agg = p.agg + static_cast<int64_t>(un.b) * p.splits * p.D;
    F2 w_in = 0, whole = kOnes;
    if (kOut) {  // what reaches the last state of the unit: ds_out through the cuts after it
      w_in = get_state(p.ds_out, un.b, c, p.D);
      for (int j = p.splits - 1; j > un.split; --j)
        w_in = through_cut(agg + static_cast<int64_t>(j) * p.D, c, p.D, w_in);
    }
    const int64_t ckpt0 = static_cast<int64_t>(un.b) * p.n_tiles;
    const Walk<kCl, true> walk(p, un, rank);
    F2 start = 0;  // the state before the tile, requested a tile ahead
    if (kOut && walk.first < un.tile1) start = get_state(p.ckpt, ckpt0 + walk.first, c, p.D);
    for (int tile = walk.first; walk.more(tile); tile += walk.step, ++round) {
      const int buffer = round & 1;
      F2 s = start;
      if (kOut && walk.more(tile + walk.step))
        start = get_state(p.ckpt, ckpt0 + tile + walk.step, c, p.D);
      if (kCl && tile >= un.tile1) {  // an empty round: w passes unchanged
        compute_barrier();  // nobody here still reads what peers may overwrite after this send
        if (warp == 0 && !dead) send(xch, round, rank, size, kOnes, 0, p.fault);
        if (!received(xch, round, ring, p)) dead = true;
        for (int j = size - 1; j >= 0; --j) {
          const ulonglong2 m = xch.of[buffer][j][l];
          w_in = fma2(m.x, w_in, m.y);
        }
        ++empty;
        continue;
      }
      const int it = kCl ? round - empty : round, st = it % p.stages;
      const uint8_t *buf = stages + st * p.stage_bytes;
      if (!mbar_wait(&ring.full[st], (it / p.stages) & 1, &ring.abort, p.status, kTimeout))
        dead = true;
      Raw qr[R], dyr[R], kr[R], vr[R];
      typename Dec::Held a[R];
      const Dec dec(p, buf + NS * kBytes, seg, l, c0);
      const uint8_t *at = buf + (seg * R * kCh + 2 * l) * static_cast<int>(sizeof(T));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int o = r * kCh * static_cast<int>(sizeof(T));
        qr[r] = *reinterpret_cast<const Raw *>(at + o);
        dyr[r] = *reinterpret_cast<const Raw *>(at + kBytes + o);
        if (kOut) {
          kr[r] = *reinterpret_cast<const Raw *>(at + 2 * kBytes + o);
          vr[r] = *reinterpret_cast<const Raw *>(at + 3 * kBytes + o);
        }
        a[r] = dec.load(r);
      }
      F2 A = kOnes, S = 0, W = 0;
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
        W = mul2(Dec::pair(a[r]), fma2(Pair<T>::f(qr[r]), Pair<T>::f(dyr[r]), W));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        A = mul2(A, Dec::pair(a[r]));
        if (kOut) S = fma2(Dec::pair(a[r]), S, mul2(Pair<T>::f(kr[r]), Pair<T>::f(vr[r])));
      }
      const F2 Ao = from_other_half(A), So = from_other_half(S), Wo = from_other_half(W);
      if (!second) {  // S through the second half, W through the first
        joint[buffer][warp][l] = make_ulonglong2(mul2(Ao, A), fma2(Ao, S, So));
        joint_w[buffer][warp][l] = fma2(A, Wo, W);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);  // every word went into A, S or W
      compute_barrier();
      F2 w = w_in, state = s;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) {  // states before each warp's rows, in order
        if (!kOut) break;
        const ulonglong2 m = joint[buffer][j][l];
        if (j == warp) s = state;
        state = fma2(m.x, state, m.y);
      }
      if constexpr (kCl) {
        // what reaches the tile's first row and this warp's last, from 0; then the round's tiles
        F2 Ap = kOnes, Wp = 0, At = kOnes, Wt = 0;
#pragma unroll
        for (int j = kWarps - 1; j >= 0; --j) {
          const F2 m = joint[buffer][j][l].x;
          if (j == warp) Ap = At, Wp = Wt;
          Wt = fma2(m, Wt, joint_w[buffer][j][l]);
          At = mul2(At, m);
        }
        if (warp == 0 && !dead) send(xch, round, rank, size, At, Wt, p.fault);
        if (!received(xch, round, ring, p)) dead = true;
#pragma unroll
        for (int j = kMaxCluster - 1; j >= 0; --j) {
          if (j >= size) continue;
          const ulonglong2 m = xch.of[buffer][j][l];
          if (j == rank) w = w_in;
          w_in = fma2(m.x, w_in, m.y);
        }
        w = fma2(Ap, w, Wp);
      } else {
#pragma unroll
        for (int j = kWarps - 1; j >= 0; --j) {  // what reaches the end of each, backwards
          const F2 m = joint[buffer][j][l].x;
          if (j == warp) w = w_in;
          w_in = fma2(m, w_in, joint_w[buffer][j][l]);
          if (!kOut) whole = mul2(whole, m);
        }
      }
      if (kOut) {
        if (second)
          s = fma2(Ao, s, So);
        else
          w = fma2(Ao, w, Wo);
        const int t0 = tile * tile_rows<C>() + seg * R;
        const Out<T, kFeed> dq(p.dq, p, un.b, t0, c, dead);
        const Out<T, kFeed> dk(p.dk, p, un.b, t0, c, dead), dv(p.dv, p, un.b, t0, c, dead);
        const Out<T, kFeed> dg(p.dg, p, un.b, t0, c, dead);  // where d_g = 1
        float sum[R];
        // apart for whole tiles, whose stores need no conditions, and for dg by single channels
        const auto gradients = [&](auto whole, auto single) {
          constexpr bool kWhole = decltype(whole)::value, kSingle = decltype(single)::value;
          F2 before[R];  // s_{t-1}
#pragma unroll
          for (int r = 0; r < R; ++r) {
            before[r] = s;
            s = fma2(Dec::pair(a[r]), s, mul2(Pair<T>::f(kr[r]), Pair<T>::f(vr[r])));
            dq.template put<kWhole>(r, mul2(Pair<T>::f(dyr[r]), s));
          }
#pragma unroll
          for (int r = R - 1; r >= 0; --r) {
            const F2 ut = fma2(Pair<T>::f(qr[r]), Pair<T>::f(dyr[r]), w);
            w = mul2(Dec::pair(a[r]), ut);
            const F2 d = mul2(w, before[r]);
            dk.template put<kWhole>(r, mul2(ut, Pair<T>::f(vr[r])));
            dv.template put<kWhole>(r, mul2(ut, Pair<T>::f(kr[r])));
            if (per_channel(kFeed)) {
              dg.template put<kWhole>(r, d);
            } else if (kSingle) {
              if (r < dg.live)
                put_state(p.dg_part, static_cast<int64_t>(un.b) * p.L + t0 + r, c, p.D, d);
            } else {
              const float2 two = unpack(d);
              sum[r] = two.x + two.y;
            }
          }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        if (!per_channel(kFeed) && p.dg_mode == 2)
          gradients(No(), Yes());
        else if (by_tma(kFeed) && dq.live >= R)
          gradients(Yes(), No());
        else
          gradients(No(), No());
        if (!per_channel(kFeed) && p.dg_mode != 2) {
          // groups of 2, 4, ..., 16 channels or whole blocks: sums over neighbouring lanes
          const int64_t row0 = static_cast<int64_t>(un.b) * p.L + t0;
          const int rows = dead ? 0 : min(R, p.L - t0);
          const int g0 = p.dg_mode == 1 ? 0 : c0 / p.d_g;
          const auto put = [&](int r, int grp, float v) {
            if (r >= rows) return;
            if (p.dg_mode == 1)
              p.dg_part[(row0 + r) * p.n_cb + un.cb] = v;
            else if (g0 + grp < p.G)
              store_one(static_cast<T *>(p.dg) + (row0 + r) * p.G + g0 + grp, v);
          };
          switch (p.d_g) {
            case 2: sum_groups<1>(sum, l, put); break;
            case 4: sum_groups<2>(sum, l, put); break;
            case 8: sum_groups<4>(sum, l, put); break;
            case 16: sum_groups<8>(sum, l, put); break;
            default: sum_groups<16>(sum, l, put);
          }
        }
      }
    }
    if (seg == 0 && !dead) {
      if (kOut && p.ds0 && un.tile0 == 0 && rank == 0) put_state(p.ds0, un.b, c, p.D, w_in);
      if (!kOut) put_cut(agg + static_cast<int64_t>(un.split) * p.D, c, p.D, whole, w_in);
    }
  }
  if (kCl) exchange_end(dead);
}

// dg of group j in a row: the sum of `width` neighbouring partial sums, in order.
template <typename T>
__global__ void __launch_bounds__(256)
    scan_dg_kernel(const float *part, T *dg, int64_t n, int width) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
    const float *s = part + i * width;
    float sum = 0.f;
    for (int j = 0; j < width; ++j) sum += s[j];
    store_one(dg + i, sum);
  }
}

// ---------------------------------------------------------------------------- one token
// One row per sequence: s_out = exp(g) s + k v, y = q s_out; s_out may be s.  VN channels per
// thread, all loads 16 bytes where the tensors allow it.  Bound: HBM (the fp32 state).
template <typename T, int VN>
__global__ void __launch_bounds__(128)
    scan_step_kernel(const T *q, const T *k, const T *v, const T *g, const float *s, T *y,
                     float *s_out, int64_t n, int D, int d_g, int G) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * VN;
  if (i >= n) return;
  const int64_t b = i / D;
  const int c = static_cast<int>(i - b * D);
  struct __align__(sizeof(T) * VN) Vt { T e[VN]; };
  struct __align__(VN >= 4 ? 16 : 4) Vf { float e[VN]; };
  const Vt qv = *reinterpret_cast<const Vt *>(q + i), kv = *reinterpret_cast<const Vt *>(k + i),
           vv = *reinterpret_cast<const Vt *>(v + i);
  Vf sv = *reinterpret_cast<const Vf *>(s + i);
  Vt yv, gv;
  const T *gr = g + b * G;
  if (d_g == 1) gv = *reinterpret_cast<const Vt *>(gr + c);
  int grp = c / d_g, left = d_g - c % d_g;  // channels of group grp from c on
  float a = d_g == 1 ? 0.f : decay(load_one(gr + grp));
#pragma unroll
  for (int e = 0; e < VN; ++e) {
    if (d_g == 1) {
      a = decay(load_one(&gv.e[e]));
    } else if (left == 0) {
      a = decay(load_one(gr + ++grp));
      left = d_g;
    }
    --left;
    sv.e[e] = fmaf(a, sv.e[e], load_one(&kv.e[e]) * load_one(&vv.e[e]));
    store_one(&yv.e[e], load_one(&qv.e[e]) * sv.e[e]);
  }
  *reinterpret_cast<Vf *>(s_out + i) = sv;
  *reinterpret_cast<Vt *>(y + i) = yv;
}

}  // namespace scan
}  // namespace hyena
