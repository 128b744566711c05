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
// Split: a CTA owns 32 channels of one sequence and walks its rows in tiles of 16 R; nothing is
// exchanged between CTAs, so the sums have one order and the result is the same in every run.
// (A row of 32 channels is 64 bytes in bf16.  At D = 4096 that gives 128 CTAs; a wider piece
// would leave most of the 148 SMs without work.)  Where a problem has too few such columns for
// the device, its time axis is cut as well: a first pass over k, v and g finds each cut's
// (A, S), and every CTA of the second pass joins those before it.
//
// Within a CTA: one warp streams the tiles in with TMA through a ring of shared-memory stages;
// eight warps compute.  Half a warp (16 lanes of 2 channels) owns a segment of R consecutive
// rows: it takes the segment into registers, frees the stage, forms the segment's (A, S), and
// after one barrier every lane joins the 16 segments of its channels in order, which gives each
// segment its own start and every warp the next tile's.  R is odd for bf16: the two halves of a
// warp then read rows an odd number of 64-byte rows apart, from different banks.
//
// All arithmetic is fp32; q, k, v, g, dy are read once, y, dq, dk, dv, dg rounded once.
// Bound: HBM bandwidth (4 flops per 8 bytes in bf16).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "ptx.cuh"

namespace hyena {
namespace scan {

constexpr int kCh = 32;               // channels of a CTA
constexpr int kSegs = 16;             // segments of a tile: 8 warps x 2 halves
constexpr int kComputeThreads = 256;
constexpr int kHelperWarps = 4;       // warp 0 of them issues TMA, 1..3 form decays (12 warps in
                                      // all: 3 per scheduler leave a thread 168 registers)
constexpr int kThreads = kComputeThreads + 32 * kHelperWarps;
constexpr int kMaxStages = 8;
constexpr unsigned int kTimeout = 1u; // HYENA_DEVICE_TIMEOUT

// How a tile's inputs reach shared memory.
enum Feed {
  kFeedChannel = 0,  // TMA, one decay per channel: g is a stream like k and v
  kFeedGroup = 1,    // TMA for the streams; the helper warps form the decays of the groups
  kFeedPlain = 2     // element loads by the helper warps (rows TMA cannot address), any d_g
};

// Rows of a tile are 16 R.  The registers of a segment and the bytes of a stage both grow with
// R; the joining of segments costs 16 steps per tile whatever R is.
template <typename T> struct Rows;
template <> struct Rows<__nv_bfloat16> { static constexpr int R = 11; };
template <> struct Rows<float> { static constexpr int R = 7; };

template <typename T>
__host__ __device__ constexpr int tile_rows() { return kSegs * Rows<T>::R; }
template <typename T>
__host__ __device__ constexpr int stream_bytes() { return tile_rows<T>() * kCh * static_cast<int>(sizeof(T)); }

struct Params {
  const void *q, *k, *v, *g, *dy;   // for kFeedPlain; g also for kFeedGroup
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
  int pieces;                       // groups a block of 32 channels touches at most
  int stages, stage_bytes;
  int dg_mode;                      // 0: dg itself, 1: one partial per block, 2: per channel
};

// ---------------------------------------------------------------------------- two channels
// One lane's two channels of a row as read from shared memory, and packed fp32 arithmetic on
// them (one instruction for both).
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  using Raw = uint32_t;
  __device__ static float2 f(Raw r) {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  __device__ static void store(__nv_bfloat16 *p, float2 x) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x.x, x.y);
    *reinterpret_cast<__nv_bfloat162 *>(p) = b;
  }
};
template <> struct Pair<float> {
  using Raw = float2;
  __device__ static float2 f(Raw r) { return r; }
  __device__ static void store(float *p, float2 x) { *reinterpret_cast<float2 *>(p) = x; }
};
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store_one(float *p, float x) { *p = x; }
__device__ __forceinline__ float load_one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_one(const float *p) { return *p; }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  mul_f32x2(d.x, d.y, a.x, a.y, b.x, b.y);
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ void compute_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory");
}

// ---------------------------------------------------------------------------- a CTA's ring
constexpr int kStageAlign = 128;  // of a TMA destination
__device__ __forceinline__ uint8_t *align_stage(uint8_t *dynamic) {
  return dynamic + (kStageAlign - smem_u32(dynamic) % kStageAlign) % kStageAlign;
}

struct Ring {
  uint64_t full[kMaxStages], empty[kMaxStages];
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

template <typename T>
__device__ __forceinline__ void fill_decays(const Params &p, float *as, int b, int c0, int t0,
                                            int thread, int threads) {
  const T *g = static_cast<const T *>(p.g) + static_cast<int64_t>(b) * p.L * p.G;
  const int g0 = c0 / p.d_g;
  for (int e = thread; e < tile_rows<T>() * p.pieces; e += threads) {
    const int row = e / p.pieces, t = t0 + row, gi = g0 + e % p.pieces;
    // rows past the end leave the state as it is
    as[e] = t < p.L && gi < p.G ? expf(load_one(g + static_cast<int64_t>(t) * p.G + gi)) : 1.0f;
  }
}

// Element loads of one stream's tile; zero outside the tensor, as TMA fills.
template <typename T>
__device__ __forceinline__ void fill_plain(const Params &p, T *dst, const void *src, int b, int c0,
                                           int t0, int thread, int threads) {
  const T *s = static_cast<const T *>(src) + static_cast<int64_t>(b) * p.L * p.D;
  for (int e = thread; e < tile_rows<T>() * kCh; e += threads) {
    const int t = t0 + e / kCh, c = c0 + e % kCh;
    dst[e] = t < p.L && c < p.D ? s[static_cast<int64_t>(t) * p.D + c] : T(0.0f);
  }
}

// The helper warps: NS streams of every tile of the CTA's units into the ring, in the order the
// compute warps take them (kReverse: last tile first).
template <typename T, int kFeed, bool kReverse, int NS>
__device__ __forceinline__ void feed(const Params &p, Ring &ring, uint8_t *stages,
                                     const CUtensorMap *const (&maps)[5],
                                     const void *const (&ptrs)[5]) {
  const int warp = threadIdx.x / 32 - kComputeThreads / 32, lane = threadIdx.x % 32;
  constexpr int kStreams = NS + (kFeed == kFeedChannel ? 1 : 0);
  constexpr int kBytes = stream_bytes<T>();
  if (kFeed == kFeedChannel && (warp != 0 || lane != 0)) return;
  if (kFeed == kFeedGroup && warp == 0 && lane != 0) return;
  int it = 0, last = 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Unit un(p, u);
    for (int i = un.tile0; i < un.tile1; ++i, ++it) {
      const int tile = kReverse ? un.tile1 - 1 - (i - un.tile0) : i;
      const int st = it % p.stages, round = it / p.stages;
      uint8_t *buf = stages + st * p.stage_bytes;
      if (round > 0 && !mbar_wait(&ring.empty[st], (round - 1) & 1, &ring.abort, p.status, kTimeout))
        goto out;
      if (kFeed != kFeedPlain && warp == 0) {
        mbar_arrive_expect_tx(&ring.full[st], kStreams * kBytes);
#pragma unroll
        for (int s = 0; s < kStreams; ++s)
          tma_load_3d(buf + s * kBytes, maps[s], &ring.full[st], un.cb * kCh,
                      tile * tile_rows<T>(), un.b);
        last = it + 1;
      }
      if (kFeed == kFeedGroup && warp > 0) {
        fill_decays<T>(p, reinterpret_cast<float *>(buf + NS * kBytes), un.b, un.cb * kCh,
                       tile * tile_rows<T>(), threadIdx.x - kComputeThreads - 32,
                       32 * (kHelperWarps - 1));
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.full[st]);
      }
      if (kFeed == kFeedPlain) {
        const int th = threadIdx.x - kComputeThreads;
#pragma unroll
        for (int s = 0; s < NS; ++s)
          fill_plain<T>(p, reinterpret_cast<T *>(buf + s * kBytes), ptrs[s], un.b, un.cb * kCh,
                        tile * tile_rows<T>(), th, 32 * kHelperWarps);
        fill_decays<T>(p, reinterpret_cast<float *>(buf + NS * kBytes), un.b, un.cb * kCh,
                       tile * tile_rows<T>(), th, 32 * kHelperWarps);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.full[st]);
      }
    }
  }
out:
  // no copy may be in flight when the CTA ends, whatever happened to the readers
  if (kFeed != kFeedPlain && warp == 0) {
    for (int j = max(0, last - p.stages); j < last; ++j) {
      int no_abort = 0;
      mbar_wait(&ring.full[j % p.stages], (j / p.stages) & 1, &no_abort, p.status, kTimeout);
    }
  }
}

template <int kFeed>
__device__ __forceinline__ void ring_init(const Params &p, Ring &ring) {
  if (threadIdx.x == 0) {
    const int arrivals = kFeed == kFeedChannel ? 1 : kHelperWarps;
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&ring.full[i], arrivals);
      mbar_init(&ring.empty[i], kComputeThreads / 32);
    }
    ring.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
}

// The decays of this lane's two channels in row r of its segment.
template <typename T, int kFeed>
struct Decays {
  const uint8_t *at;  // kFeedChannel: the lane's g pair in its segment's first row; else the rows
                      // of fp32 decays
  int pieces, i0, i1;
  __device__ float2 operator()(int r) const {
    if (kFeed == kFeedChannel) {
      const float2 g = Pair<T>::f(*reinterpret_cast<const typename Pair<T>::Raw *>(
          at + r * kCh * static_cast<int>(sizeof(T))));
      return make_float2(expf(g.x), expf(g.y));
    }
    const float *a = reinterpret_cast<const float *>(at) + r * pieces;
    return make_float2(a[i0], a[i1]);
  }
};

template <typename T, int kFeed>
__device__ __forceinline__ Decays<T, kFeed> decays_at(const Params &p, const uint8_t *streams_end,
                                                      int seg, int l, int c0) {
  Decays<T, kFeed> d;
  constexpr int R = Rows<T>::R;
  if (kFeed == kFeedChannel) {
    d.at = streams_end + (seg * R * kCh + 2 * l) * static_cast<int>(sizeof(T));
    d.pieces = d.i0 = d.i1 = 0;
  } else {
    const int g0 = c0 / p.d_g, c = c0 + 2 * l;
    d.at = streams_end + seg * R * p.pieces * 4;
    d.pieces = p.pieces;
    d.i0 = min(c, p.D - 1) / p.d_g - g0;
    d.i1 = min(c + 1, p.D - 1) / p.d_g - g0;
  }
  return d;
}

// Stores a lane's two channels of one row (nothing outside the tensor).
template <typename T, int kFeed>
__device__ __forceinline__ void put(T *row, int c, int D, float2 x) {
  if (kFeed != kFeedPlain) {  // D is a multiple of 16 bytes: a pair is inside or outside
    if (c < D) Pair<T>::store(row + c, x);
  } else {
    if (c < D) store_one(row + c, x.x);
    if (c + 1 < D) store_one(row + c + 1, x.y);
  }
}

__device__ __forceinline__ float2 get_state(const float *s, int64_t row, int c, int D) {
  if (!s) return make_float2(0.f, 0.f);
  s += row * D;
  return make_float2(c < D ? s[c] : 0.f, c + 1 < D ? s[c + 1] : 0.f);
}
__device__ __forceinline__ void put_state(float *s, int64_t row, int c, int D, float2 x) {
  s += row * D;
  if (c < D) s[c] = x.x;
  if (c + 1 < D) s[c + 1] = x.y;
}

// ---------------------------------------------------------------------------- forward
// kOut: y and the last state (streams k, v, q); otherwise only states: checkpoints, or the (A, S)
// of the unit's time cut from a zero state (streams k, v).
template <typename T, int kFeed, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    scan_fwd_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                    const Params p) {
  extern __shared__ uint8_t dynamic[];
  uint8_t *stages = align_stage(dynamic);
  __shared__ Ring ring;
  __shared__ float4 joint[2][kSegs][kCh / 2];  // (A, A, S, S) of a segment's two channels
  constexpr int R = Rows<T>::R, NS = kOut ? 3 : 2, kBytes = stream_bytes<T>();
  using Raw = typename Pair<T>::Raw;
  ring_init<kFeed>(p, ring);
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x >= kComputeThreads) {
    const CUtensorMap *const maps[5] = {&mk, &mv, kOut ? &mq : &mg, &mg, nullptr};
    const void *const ptrs[5] = {p.k, p.v, p.q, nullptr, nullptr};
    feed<T, kFeed, false, NS>(p, ring, stages, maps, ptrs);
    return;
  }
  const int lane = threadIdx.x % 32, l = lane % 16, seg = threadIdx.x / 16;
  bool dead = false;
  int it = 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Unit un(p, u);
    const int c0 = un.cb * kCh, c = c0 + 2 * l;
    // the state before the unit: s0 through the cuts before it
    float2 carry = make_float2(0.f, 0.f), whole = make_float2(1.f, 1.f);
    if (kOut || !p.agg || p.ckpt) {
      carry = get_state(p.s0, un.b, c, p.D);
      if (p.agg)
        for (int j = 0; j < un.split; ++j) {
          const float2 *ag = p.agg + (static_cast<int64_t>(un.b) * p.splits + j) * p.D;
          if (c < p.D) carry.x = fmaf(ag[c].x, carry.x, ag[c].y);
          if (c + 1 < p.D) carry.y = fmaf(ag[c + 1].x, carry.y, ag[c + 1].y);
        }
    }
    for (int tile = un.tile0; tile < un.tile1; ++tile, ++it) {
      const int st = it % p.stages;
      const uint8_t *buf = stages + st * p.stage_bytes;
      if (!mbar_wait(&ring.full[st], (it / p.stages) & 1, &ring.abort, p.status, kTimeout))
        dead = true;
      float2 x[R], a[R];
      Raw qr[R];
      const Decays<T, kFeed> dec = decays_at<T, kFeed>(p, buf + NS * kBytes, seg, l, c0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int at = ((seg * R + r) * kCh + 2 * l) * static_cast<int>(sizeof(T));
        x[r] = mul2(Pair<T>::f(*reinterpret_cast<const Raw *>(buf + at)),
                    Pair<T>::f(*reinterpret_cast<const Raw *>(buf + kBytes + at)));
        if (kOut) qr[r] = *reinterpret_cast<const Raw *>(buf + 2 * kBytes + at);
        a[r] = dec(r);
      }
      float2 A = a[0], S = x[0];
#pragma unroll
      for (int r = 1; r < R; ++r) {
        S = fma2(a[r], S, x[r]);
        A = mul2(A, a[r]);
      }
      joint[it & 1][seg][l] = make_float4(A.x, A.y, S.x, S.y);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);  // the segment is in registers
      compute_barrier();
      if (p.ckpt && seg == 0 && !dead)
        put_state(p.ckpt, static_cast<int64_t>(un.b) * p.n_tiles + tile, c, p.D, carry);
      float2 s = carry;
#pragma unroll
      for (int j = 0; j < kSegs; ++j) {
        const float4 m = joint[it & 1][j][l];
        if (j == seg) s = carry;
        carry = fma2(make_float2(m.x, m.y), carry, make_float2(m.z, m.w));
        if (!kOut) whole = mul2(whole, make_float2(m.x, m.y));
      }
      if (kOut && !dead) {
        const int t0 = tile * tile_rows<T>() + seg * R;
        T *row = static_cast<T *>(p.y) + (static_cast<int64_t>(un.b) * p.L + t0) * p.D;
        const int rows = min(R, p.L - t0);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s = fma2(a[r], s, x[r]);
          if (r < rows) put<T, kFeed>(row + static_cast<int64_t>(r) * p.D, c, p.D,
                                      mul2(Pair<T>::f(qr[r]), s));
        }
      }
    }
    if (seg == 0 && !dead) {
      if (p.s_out && un.tile1 == p.n_tiles) put_state(p.s_out, un.b, c, p.D, carry);
      if (!kOut && p.agg && !p.ckpt) {
        float2 *ag = p.agg + (static_cast<int64_t>(un.b) * p.splits + un.split) * p.D;
        if (c < p.D) ag[c] = make_float2(whole.x, carry.x);
        if (c + 1 < p.D) ag[c + 1] = make_float2(whole.y, carry.y);
      }
    }
  }
}

// ---------------------------------------------------------------------------- backward
// kOut: the gradients (streams q, dy, k, v and the checkpoints); otherwise the (A, W) of the
// unit's time cut from w = 0 (streams q, dy).
template <typename T, int kFeed, bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    scan_bwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mdy,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap mg, const Params p) {
  extern __shared__ uint8_t dynamic[];
  uint8_t *stages = align_stage(dynamic);
  __shared__ Ring ring;
  __shared__ float4 joint[2][kSegs][kCh / 2];   // (A, A, S, S)
  __shared__ float2 joint_w[2][kSegs][kCh / 2];
  constexpr int R = Rows<T>::R, NS = kOut ? 4 : 2, kBytes = stream_bytes<T>();
  using Raw = typename Pair<T>::Raw;
  ring_init<kFeed>(p, ring);
  griddep_launch_dependents();
  griddep_wait();
  if (threadIdx.x >= kComputeThreads) {
    const CUtensorMap *const maps[5] = {&mq, &mdy, kOut ? &mk : &mg, &mv, &mg};
    const void *const ptrs[5] = {p.q, p.dy, p.k, p.v, nullptr};
    feed<T, kFeed, true, NS>(p, ring, stages, maps, ptrs);
    return;
  }
  const int lane = threadIdx.x % 32, l = lane % 16, seg = threadIdx.x / 16;
  bool dead = false;
  int it = 0;
  for (int u = blockIdx.x; u < p.n_units; u += gridDim.x) {
    const Unit un(p, u);
    const int c0 = un.cb * kCh, c = c0 + 2 * l;
    // what reaches the last state of the unit: ds_out through the cuts after it
    float2 w_in = make_float2(0.f, 0.f), whole = make_float2(1.f, 1.f);
    if (kOut) {
      w_in = get_state(p.ds_out, un.b, c, p.D);
      for (int j = p.splits - 1; j > un.split; --j) {
        const float2 *ag = p.agg + (static_cast<int64_t>(un.b) * p.splits + j) * p.D;
        if (c < p.D) w_in.x = fmaf(ag[c].x, w_in.x, ag[c].y);
        if (c + 1 < p.D) w_in.y = fmaf(ag[c + 1].x, w_in.y, ag[c + 1].y);
      }
    }
    for (int tile = un.tile1 - 1; tile >= un.tile0; --tile, ++it) {
      const int st = it % p.stages;
      const uint8_t *buf = stages + st * p.stage_bytes;
      float2 s = make_float2(0.f, 0.f);
      if (kOut) s = get_state(p.ckpt, static_cast<int64_t>(un.b) * p.n_tiles + tile, c, p.D);
      if (!mbar_wait(&ring.full[st], (it / p.stages) & 1, &ring.abort, p.status, kTimeout))
        dead = true;
      Raw qr[R], dyr[R], kr[R], vr[R];
      float2 a[R];
      const Decays<T, kFeed> dec = decays_at<T, kFeed>(p, buf + NS * kBytes, seg, l, c0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int at = ((seg * R + r) * kCh + 2 * l) * static_cast<int>(sizeof(T));
        qr[r] = *reinterpret_cast<const Raw *>(buf + at);
        dyr[r] = *reinterpret_cast<const Raw *>(buf + kBytes + at);
        if (kOut) {
          kr[r] = *reinterpret_cast<const Raw *>(buf + 2 * kBytes + at);
          vr[r] = *reinterpret_cast<const Raw *>(buf + 3 * kBytes + at);
        }
        a[r] = dec(r);
      }
      float2 A = make_float2(1.f, 1.f), S = make_float2(0.f, 0.f), W = S;
#pragma unroll
      for (int r = R - 1; r >= 0; --r)
        W = mul2(a[r], fma2(Pair<T>::f(qr[r]), Pair<T>::f(dyr[r]), W));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        A = mul2(A, a[r]);
        if (kOut) S = fma2(a[r], S, mul2(Pair<T>::f(kr[r]), Pair<T>::f(vr[r])));
      }
      joint[it & 1][seg][l] = make_float4(A.x, A.y, S.x, S.y);
      joint_w[it & 1][seg][l] = W;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[st]);
      compute_barrier();
      float2 w = w_in, sj = s;
#pragma unroll
      for (int j = 0; j < kSegs; ++j) {  // states before each segment, in order
        const float4 m = joint[it & 1][j][l];
        if (j == seg) s = sj;
        if (kOut) sj = fma2(make_float2(m.x, m.y), sj, make_float2(m.z, m.w));
      }
#pragma unroll
      for (int j = kSegs - 1; j >= 0; --j) {  // what reaches the end of each, backwards
        const float4 m = joint[it & 1][j][l];
        if (j == seg) w = w_in;
        w_in = fma2(make_float2(m.x, m.y), w_in, joint_w[it & 1][j][l]);
        if (!kOut) whole = mul2(whole, make_float2(m.x, m.y));
      }
      if (kOut) {
        const int t0 = tile * tile_rows<T>() + seg * R;
        const int rows = min(R, p.L - t0);
        const int64_t row0 = static_cast<int64_t>(un.b) * p.L + t0;
        float2 before[R];  // s_{t-1}
#pragma unroll
        for (int r = 0; r < R; ++r) {
          before[r] = s;
          const float2 k = Pair<T>::f(kr[r]), v = Pair<T>::f(vr[r]);
          s = fma2(a[r], s, mul2(k, v));
          if (r < rows && !dead)
            put<T, kFeed>(static_cast<T *>(p.dq) + (row0 + r) * p.D, c, p.D,
                          mul2(Pair<T>::f(dyr[r]), s));
        }
#pragma unroll
        for (int r = R - 1; r >= 0; --r) {
          const float2 un_t = fma2(Pair<T>::f(qr[r]), Pair<T>::f(dyr[r]), w);
          w = mul2(a[r], un_t);
          const float2 dg = mul2(w, before[r]);
          const bool live = r < rows && !dead;
          if (live) {
            put<T, kFeed>(static_cast<T *>(p.dk) + (row0 + r) * p.D, c, p.D,
                          mul2(un_t, Pair<T>::f(vr[r])));
            put<T, kFeed>(static_cast<T *>(p.dv) + (row0 + r) * p.D, c, p.D,
                          mul2(un_t, Pair<T>::f(kr[r])));
          }
          if (kFeed == kFeedChannel || p.d_g == 1) {
            if (live) put<T, kFeed>(static_cast<T *>(p.dg) + (row0 + r) * p.D, c, p.D, dg);
          } else if (p.dg_mode == 2) {
            if (live) put_state(p.dg_part, row0 + r, c, p.D, dg);
          } else {
            // groups of 2, 4, ..., 16 channels, or whole blocks: a sum over neighbouring lanes
            const int span = min(p.d_g, kCh) / 2;
            float sum = dg.x + dg.y;
            for (int o = 1; o < span; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (live && c < p.D && l % span == 0) {
              if (p.dg_mode == 1)
                p.dg_part[(row0 + r) * p.n_cb + un.cb] = sum;
              else
                store_one(static_cast<T *>(p.dg) + (row0 + r) * p.G + c / p.d_g, sum);
            }
          }
        }
      }
    }
    if (seg == 0 && !dead) {
      if (kOut && p.ds0 && un.tile0 == 0) put_state(p.ds0, un.b, c, p.D, w_in);
      if (!kOut) {
        float2 *ag = p.agg + (static_cast<int64_t>(un.b) * p.splits + un.split) * p.D;
        if (c < p.D) ag[c] = make_float2(whole.x, w_in.x);
        if (c + 1 < p.D) ag[c + 1] = make_float2(whole.y, w_in.y);
      }
    }
  }
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
  float a = d_g == 1 ? 0.f : expf(load_one(gr + grp));
#pragma unroll
  for (int e = 0; e < VN; ++e) {
    if (d_g == 1) {
      a = expf(load_one(&gv.e[e]));
    } else if (left == 0) {
      a = expf(load_one(gr + ++grp));
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
