// hyena_scan.cu -- host side of the gated linear recurrence (include/hyena_mixer.h): argument
// checks, time cuts, TMA descriptors and launches of the kernels in scan.cuh.
#include <algorithm>
#include <cstdint>
#include <limits>
#include <mutex>

#include "host_util.h"
#include "hyena_conv_testing.h"
#include "hyena_mixer.h"
#include "scan.cuh"

namespace {

namespace sc = hyena::scan;
using hyena::host::aligned;
using hyena::host::overlap;
using hyena::host::round_up;

constexpr int kSmemMax = 227 * 1024;
constexpr int kCopySmem = 148 * 1024;   // where tiles come by copies (see plan)
constexpr int kStaticSmem = 16 * 1024;  // bound on a kernel's static shared memory
constexpr int64_t kI32 = std::numeric_limits<int32_t>::max();

struct Shape {
  int64_t B, L, D;
  int d_g, dtype;
  int64_t es() const { return dtype == HYENA_DTYPE_F32 ? 4 : 2; }
  int64_t G() const { return D / d_g; }
  int64_t n_cb() const { return (D + sc::kCh - 1) / sc::kCh; }
  int64_t rows() const {
    return dtype == HYENA_DTYPE_F32 ? sc::tile_rows<sc::F32>() : sc::tile_rows<sc::Bf16>();
  }
  int64_t n_tiles() const { return (L + rows() - 1) / rows(); }
  int64_t numel() const { return B * L * D; }
};

int check_shape(const Shape &s) {
  if (s.dtype != HYENA_DTYPE_BF16 && s.dtype != HYENA_DTYPE_F32) return HYENA_ERR_INVALID_ARG;
  if (s.B < 0 || s.L < 0 || s.D < 1 || s.d_g < 1 || s.D % s.d_g != 0) return HYENA_ERR_INVALID_ARG;
  if (s.B > kI32 || s.L > kI32 - 4096 || s.D > (int64_t{1} << 28)) return HYENA_ERR_INVALID_ARG;
  if (s.B == 0) return HYENA_OK;
  const int64_t lim = std::numeric_limits<int64_t>::max() / 64;
  const int64_t l = std::max<int64_t>(s.L, 1);
  if (s.B > lim / l || s.B * l > lim / s.D) return HYENA_ERR_INVALID_ARG;
  return HYENA_OK;
}

// How the time axis of a column of 32 channels is shared, where there are too few columns for the
// device (a CTA streams ~50 GB/s at best): by a cluster whose CTAs take neighbouring tiles and tell
// each other their (A, S), round by round, or by cuts, whose (A, S) a first pass over k, v and g
// finds; that reaches more CTAs, but costs a launch and reads three of the five streams again.  The
// constants are us a tile, from both sides' measurements of bf16 forwards:
//                              alone   cluster    cuts
//   [1, 8192, 2048], d_g 64     46.2      35.5    47.1
//   [2, 5000, 512],  d_g 64     29.2      14.1    19.7
//   [1, 65536, 496], d_g 1     386.7     104.6   105.1   (backward 825.7, 168.3, 151.1)
//   [1, 65536, 500], d_g 1     519.0     135.0   116.8   (backward 1454, 271.0, 224.1)
//   [1, 65536, 498], d_g 2      1855     318.2   404.8   (rows by single elements)
struct Cuts {
  int splits, tiles_per_split, cluster;
};
Cuts cuts_of(const Shape &s) {
  constexpr int64_t kCtas = 148;
  constexpr double kTile = 1.0, kExchange = 0.7, kLaunch = 6.0;
  const double two_passes = s.D * s.es() % 8 == 0 ? 2.4 : 3.2;
  // clusters of so many CTAs that run at once, a little below what the occupancy query answers (74,
  // 45, 33, 26, 22, 15, 15), since it varies with the SMs that a GPC has
  constexpr int kClusters[sc::kMaxCluster + 1] = {0, 148, 72, 44, 32, 24, 20, 14, 14};
  const int64_t blocks = s.B * s.n_cb(), tiles = s.n_tiles();
  Cuts best{1, static_cast<int>(tiles), 1};
  if (blocks * 2 > kCtas) return best;
  double best_us = static_cast<double>(tiles) * kTile;
  for (int n = 2; n <= sc::kMaxCluster && n <= tiles; ++n) {
    const int64_t waves = (blocks + kClusters[n] - 1) / kClusters[n];
    const double us = static_cast<double>(waves) *
                      (static_cast<double>((tiles + n - 1) / n) * (kTile + kExchange) + 1.0);
    if (us < best_us) {
      best_us = us;
      best = Cuts{1, static_cast<int>(tiles), n};
    }
  }
  const int64_t want = std::min(kCtas / blocks, tiles / 2);
  if (want > 1) {
    const int64_t per = (tiles + want - 1) / want;
    if (static_cast<double>(per) * two_passes + kLaunch < best_us)
      best = Cuts{static_cast<int>((tiles + per - 1) / per), static_cast<int>(per), 1};
  }
  return best;
}

int64_t agg_bytes(const Shape &s) {
  const int64_t n = cuts_of(s).splits;
  return n > 1 ? round_up(s.B * n * s.D * 8, 256) : 0;
}
int64_t ckpt_bytes(const Shape &s) { return round_up(s.B * s.n_tiles() * s.D * 4, 256); }

int dg_mode(const Shape &s) {
  if (s.d_g <= sc::kCh && (s.d_g & (s.d_g - 1)) == 0) return 0;
  return s.d_g % sc::kCh == 0 ? 1 : 2;
}
int64_t dg_bytes(const Shape &s) {
  const int m = dg_mode(s);
  return m == 0 ? 0 : round_up(s.B * s.L * (m == 1 ? s.n_cb() : s.D) * 4, 256);
}

// How the groups' rows of g arrive: a tile from a multiple of g_align groups at or before a block's
// first group to its last.
void choose_groups(const Shape &s, const void *g, sc::Params *p) {
  const int per16 = static_cast<int>(16 / s.es()), per4 = static_cast<int>(4 / s.es());
  p->g_feed = s.G() % per16 == 0 && aligned(g, 16) ? sc::kGroupsTma
              : s.G() % per4 == 0 && aligned(g, 4) ? sc::kGroupsCopy
                                                   : sc::kGroupsElement;
  p->g_align = p->g_feed == sc::kGroupsTma ? per16 : p->g_feed == sc::kGroupsCopy ? per4 : 1;
  // blocks of 32 channels start at every pieces-th group where those are whole
  const bool whole = s.d_g % sc::kCh == 0 || sc::kCh % s.d_g == 0;
  const bool fits = whole && (p->pieces % p->g_align == 0 || p->g_align % p->pieces == 0);
  p->g_box = static_cast<int>(round_up(fits ? p->pieces : p->pieces + p->g_align - 1, p->g_align));
  while ((1 << p->copy_bits) * per4 < p->g_box) ++p->copy_bits;
}

// One tensor [B, L, width] as boxes of `box_w` columns and one tile's rows.
int encode(CUtensorMap *m, const Shape &s, const void *ptr, int64_t width, int box_w) {
  hyena::host::EncodeTiledFn enc = hyena::host::encode_tiled();
  if (!enc) return HYENA_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(s.L),
                              static_cast<cuuint64_t>(s.B)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(width * s.es()),
                                 static_cast<cuuint64_t>(s.L * width * s.es())};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_w), static_cast<cuuint32_t>(s.rows()), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const auto type = s.dtype == HYENA_DTYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(m, type, 3, const_cast<void *>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

int encode(CUtensorMap *m, const Shape &s, const void *ptr) {
  return encode(m, s, ptr, s.D, sc::kCh);
}

template <typename F>
void allow(F *kernel, cudaError_t *e) {
  if (*e == cudaSuccess)
    *e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax - kStaticSmem);
}
// A kernel that moves registers between its warps waits for ever if it starts with fewer than it
// counts on, so what it was compiled to is looked up.
template <typename F>
void allow_registers(F *kernel, cudaError_t *e) {
  cudaFuncAttributes a{};
  if (*e == cudaSuccess) *e = cudaFuncGetAttributes(&a, reinterpret_cast<const void *>(kernel));
  if (*e == cudaSuccess && a.numRegs < sc::kStartRegs) *e = cudaErrorInvalidConfiguration;
}
template <typename C, int kFeed>
void allow_smem(cudaError_t *e) {
  allow(sc::scan_fwd_kernel<C, kFeed, true, false>, e);
  allow(sc::scan_fwd_kernel<C, kFeed, true, true>, e);
  allow(sc::scan_fwd_kernel<C, kFeed, false, false>, e);
  if constexpr (kFeed != sc::kTmaRaw || sizeof(typename C::T) == 2) {
    allow(sc::scan_fwd_kernel<C, kFeed, false, true>, e);
    allow(sc::scan_bwd_kernel<C, kFeed, true, false>, e);
    allow(sc::scan_bwd_kernel<C, kFeed, true, true>, e);
    allow_registers(sc::scan_bwd_kernel<C, kFeed, true, false>, e);
    allow_registers(sc::scan_bwd_kernel<C, kFeed, true, true>, e);
    allow(sc::scan_bwd_kernel<C, kFeed, false, false>, e);
  }
}

// f(integral constant) for every feed.
template <typename F>
void with_feed(F &&f) {
  f(std::integral_constant<int, sc::kTmaChannel>());
  f(std::integral_constant<int, sc::kTmaGroup>());
  f(std::integral_constant<int, sc::kCopyChannel>());
  f(std::integral_constant<int, sc::kCopyGroup>());
  f(std::integral_constant<int, sc::kTmaRaw>());
}

// Per-device one-time opt-in to the kernels' shared memory.
int prepare_device(hyena::host::DeviceInfo *info) {
  if (hyena::host::device_info(info) != HYENA_OK) return HYENA_ERR_CUDA;
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return HYENA_ERR_CUDA;
  std::call_once(once[dev], [dev]() {
    cudaError_t e = cudaSuccess;
    with_feed([&](auto feed) {
      allow_smem<sc::F32, decltype(feed)::value>(&e);
      allow_smem<sc::Bf16, decltype(feed)::value>(&e);
    });
    err[dev] = e;
  });
  return err[dev] == cudaSuccess ? HYENA_OK : HYENA_ERR_CUDA;
}

sc::Params base_params(const Shape &s, const void *g, const hyena::host::DeviceInfo &info) {
  sc::Params p{};
  const Cuts c = cuts_of(s);
  p.status = info.status;
  p.wait_ns = hyena::kWaitTimeoutNs;
  p.B = static_cast<int>(s.B);
  p.L = static_cast<int>(s.L);
  p.D = static_cast<int>(s.D);
  p.d_g = s.d_g;
  p.G = static_cast<int>(s.G());
  p.n_cb = static_cast<int>(s.n_cb());
  p.n_tiles = static_cast<int>(s.n_tiles());
  p.splits = c.splits;
  p.tiles_per_split = c.tiles_per_split;
  p.cluster = c.cluster;
  p.pieces = s.d_g % sc::kCh == 0   ? 1
             : sc::kCh % s.d_g == 0 ? sc::kCh / s.d_g
                                    : (sc::kCh + s.d_g - 2) / s.d_g + 1;
  while ((1 << p.piece_bits) < p.pieces) ++p.piece_bits;
  p.dg_mode = dg_mode(s);
  if (s.d_g > 1) choose_groups(s, g, &p);
  return p;
}

// Cuts [first, first + count) of the problem with `streams` tiles per stage (and the decays).
struct Launch {
  unsigned grid;
  size_t smem;
};
template <typename C>
Launch plan(sc::Params &p, int feed, int streams, int first, int count, int sm_count) {
  int decays = sc::stream_bytes<C>();  // a stream of g, or decays and the groups' rows of g
  if (!sc::per_channel(feed)) {
    decays = feed == sc::kTmaGroup ? sc::decay_bytes<C>(p.pieces) : 0;
    if (feed != sc::kTmaGroup || p.g_feed != sc::kGroupsElement)
      decays += static_cast<int>(round_up(
          sc::tile_rows<C>() * p.g_box * static_cast<int64_t>(sizeof(typename C::T)), sc::kStageAlign));
  }
  p.stage_bytes = streams * sc::stream_bytes<C>() + decays;
  // Copies on their way to shared memory hold lines of the L1 cache, which shares its memory: with
  // all of it given to the ring ~9 KB were in flight and the forward of L = 65536, D = 500 took
  // 236 us; with rings of 80 to 180 KB 118 us (D = 496, by TMA: 105).
  const bool all_tma = sc::by_tma(feed) && (sc::per_channel(feed) || p.g_feed == sc::kGroupsTma);
  const int room = (all_tma ? kSmemMax : kCopySmem) - kStaticSmem - sc::kStageAlign;
  p.stages = std::max(2, std::min(sc::kMaxStages, room / p.stage_bytes));
  p.unit_split0 = first;
  p.unit_splits = count;
  p.n_units = p.B * count * p.n_cb;
  Launch l;
  l.grid = static_cast<unsigned>(p.cluster > 1 ? p.n_units * p.cluster : std::min(p.n_units, sm_count));
  l.smem = static_cast<size_t>(p.stages) * p.stage_bytes + sc::kStageAlign;
  return l;
}

template <typename C, int kFeed, bool kOut, bool kCl>
int run_fwd(const Shape &s, sc::Params p, int first, int count, int sms, cudaStream_t stream) {
  const Launch l = plan<C>(p, kFeed, kOut ? 3 : 2, first, count, sms);
  CUtensorMap mk{}, mv{}, mq{}, mg{};
  if (sc::by_tma(kFeed)) {
    if (encode(&mk, s, p.k) || encode(&mv, s, p.v) || (kOut && encode(&mq, s, p.q)) ||
        (kFeed == sc::kTmaChannel && encode(&mg, s, p.g)) ||
        (s.d_g > 1 && p.g_feed == sc::kGroupsTma && encode(&mg, s, p.g, s.G(), p.g_box)))
      return HYENA_ERR_CUDA;
  }
  return hyena::host::launch_in_clusters(
             kCl ? p.cluster : 1, sc::scan_fwd_kernel<C, kFeed, kOut, kCl>, dim3(l.grid),
                             dim3(sc::kThreads), l.smem, stream, mk, mv, mq, mg,
                             p) == cudaSuccess
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

template <typename C, int kFeed, bool kOut, bool kCl>
int run_bwd(const Shape &s, sc::Params p, int first, int count, int sms, cudaStream_t stream) {
  const Launch l = plan<C>(p, kFeed, kOut ? 4 : 2, first, count, sms);
  CUtensorMap mq{}, mdy{}, mk{}, mv{}, mg{};
  if (sc::by_tma(kFeed)) {
    if (encode(&mq, s, p.q) || encode(&mdy, s, p.dy) || (kOut && encode(&mk, s, p.k)) ||
        (kOut && encode(&mv, s, p.v)) || (kFeed == sc::kTmaChannel && encode(&mg, s, p.g)) ||
        (s.d_g > 1 && p.g_feed == sc::kGroupsTma && encode(&mg, s, p.g, s.G(), p.g_box)))
      return HYENA_ERR_CUDA;
  }
  return hyena::host::launch_in_clusters(
             kCl ? p.cluster : 1, sc::scan_bwd_kernel<C, kFeed, kOut, kCl>, dim3(l.grid),
                             dim3(sc::kThreads), l.smem, stream, mq, mdy, mk, mv, mg,
                             p) == cudaSuccess
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

// The states pass over the whole problem: y and the last state, or (kOut = false) checkpoints.
template <typename C, int kFeed, bool kOut>
int states(const Shape &s, sc::Params p, float2 *agg, int sms, cudaStream_t stream) {
  if (p.splits > 1) {
    sc::Params a = p;
    a.agg = agg;
    a.ckpt = nullptr;
    a.s_out = nullptr;
    const int rc = run_fwd<C, kFeed, false, false>(s, a, 0, p.splits - 1, sms, stream);
    if (rc != HYENA_OK) return rc;
    p.agg = agg;
  }
  if (p.cluster > 1) return run_fwd<C, kFeed, kOut, true>(s, p, 0, 1, sms, stream);
  return run_fwd<C, kFeed, kOut, false>(s, p, 0, p.splits, sms, stream);
}

template <typename C, int kFeed>
int forward(const Shape &s, const sc::Params &p, void *ws, int sms, cudaStream_t stream) {
  return states<C, kFeed, true>(s, p, static_cast<float2 *>(ws), sms, stream);
}

template <typename C, int kFeed>
int backward(const Shape &s, sc::Params p, void *ws, int sms, cudaStream_t stream) {
  uint8_t *at = static_cast<uint8_t *>(ws);
  float2 *agg = reinterpret_cast<float2 *>(at);
  at += agg_bytes(s);
  p.dg_part = reinterpret_cast<float *>(at);
  at += dg_bytes(s);
  int rc = HYENA_OK;
  if (!p.ckpt) {
    p.ckpt = reinterpret_cast<float *>(at);
    rc = states<C, kFeed, false>(s, p, agg, sms, stream);
    if (rc != HYENA_OK) return rc;
  }
  if (p.splits > 1) {
    p.agg = agg;
    rc = run_bwd<C, kFeed, false, false>(s, p, 1, p.splits - 1, sms, stream);
    if (rc != HYENA_OK) return rc;
  }
  rc = p.cluster > 1 ? run_bwd<C, kFeed, true, true>(s, p, 0, 1, sms, stream)
                     : run_bwd<C, kFeed, true, false>(s, p, 0, p.splits, sms, stream);
  if (rc != HYENA_OK || p.dg_mode == 0) return rc;
  const int64_t n = s.B * s.L * s.G();
  const int width = p.dg_mode == 1 ? s.d_g / sc::kCh : s.d_g;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 16 * sms));
  return hyena::host::launch(sc::scan_dg_kernel<typename C::T>, dim3(grid), dim3(256), 0, stream,
                             static_cast<const float *>(p.dg_part), static_cast<typename C::T *>(p.dg), n,
                             width) == cudaSuccess
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

// Which feed takes the tensors, from their rows and addresses; sets the copies' and stores' width.
// TMA needs rows and bases of 16 bytes, and a group's decay for both channels of a pair.  The
// compute warps take the exps of groups up to `raw` channels, the helpers those of wider ones, whose
// few exps the compute warps need not repeat.  L = 8192, D = 4096, by compute warps | by helpers, us:
//   d_g                   2            4            8           16           64
//   forward, bf16    52 | 127     50 |  85     50 |  78     49 |  50     50 |  48
//   forward, fp32    99 | 121     93 | 108     89 | 102     89 |  88     88 |  87
//   backward, bf16  132 | 163    122 | 118
//   backward, fp32  203 | 174    158 | 159
// (forward, d_g = 8, fp32, B = 8, L = 4096: 364 | 353, the one shape of five that went the other way)
int choose_feed(const Shape &s, std::initializer_list<const void *> streams,
                std::initializer_list<const void *> outs, const void *g, int raw, sc::Params *p) {
  uintptr_t bits = static_cast<uintptr_t>(s.D * s.es()), out_bits = bits;
  for (const void *t : streams) bits |= reinterpret_cast<uintptr_t>(t);
  if (s.d_g == 1) bits |= reinterpret_cast<uintptr_t>(g);
  for (const void *t : outs) out_bits |= reinterpret_cast<uintptr_t>(t);
  const uintptr_t pair = static_cast<uintptr_t>(2 * s.es());
  p->pair_out = out_bits % pair == 0;
  p->copy = bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 0;
  const bool tma = bits % 16 == 0 && p->pair_out && s.D * s.es() * s.L < (int64_t{1} << 40) &&
                   (s.d_g == 1 || s.d_g % 2 == 0);
  return tma ? (s.d_g == 1                                        ? sc::kTmaChannel
                : s.d_g <= raw && p->g_feed != sc::kGroupsElement ? sc::kTmaRaw
                                                                  : sc::kTmaGroup)
             : (s.d_g == 1 ? sc::kCopyChannel : sc::kCopyGroup);
}

template <typename F>
int with_one_feed(int feed, F &&f) {
  int rc = HYENA_ERR_UNSUPPORTED;
  with_feed([&](auto one) {
    if (decltype(one)::value == feed) rc = f(one);
  });
  return rc;
}

// Copies a state (zeros if null) for problems of no tokens.
int copy_state(const float *from, float *to, int64_t n, cudaStream_t stream) {
  if (!to || n == 0) return HYENA_OK;
  const size_t bytes = static_cast<size_t>(n) * 4;
  const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(to, 0, bytes, stream);
  return e == cudaSuccess ? HYENA_OK : HYENA_ERR_CUDA;
}

struct Buf {
  const void *p;
  int64_t bytes;
};
// Whether an output overlaps an input or another output.
bool clash(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf *o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf &i : ins)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return true;
    for (const Buf *q = o + 1; q != outs.end(); ++q)
      if (overlap(o->p, o->bytes, q->p, q->bytes)) return true;
  }
  return false;
}

bool misaligned(uintptr_t a, std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs)
    if (!aligned(p, a)) return true;
  return false;
}

// hyena_scan_fwd with the test settings of hyena_testing_scan_fault (0, 0 in the product path).
int scan_fwd(const void *q, const void *k, const void *v, const void *g, const float *s0, void *y,
             float *s_out, float *ckpt, int64_t B, int64_t L, int64_t D, int d_g, int dtype,
             void *workspace, size_t workspace_bytes, int fault, uint64_t wait_ns,
             cudaStream_t stream) {
  const Shape s{B, L, D, d_g, dtype};
  int rc = check_shape(s);
  if (rc != HYENA_OK) return rc;
  if (misaligned(4, {s0, s_out, ckpt})) return HYENA_ERR_MISALIGNED;
  if (B == 0) return HYENA_OK;
  const int64_t st = B * D * 4, n = s.numel() * s.es(), ng = B * L * s.G() * s.es();
  if (overlap(s_out, st, s0, st)) return HYENA_ERR_INVALID_ARG;
  if (L == 0) return copy_state(s0, s_out, B * D, stream);
  if (!q || !k || !v || !g || !y) return HYENA_ERR_INVALID_ARG;
  if (misaligned(static_cast<uintptr_t>(s.es()), {q, k, v, g, y}) || !aligned(workspace, 16))
    return HYENA_ERR_MISALIGNED;
  const int64_t need = agg_bytes(s);
  if (need > 0 && (!workspace || static_cast<int64_t>(workspace_bytes) < need))
    return HYENA_ERR_INVALID_ARG;
  const int64_t nck = ckpt ? B * s.n_tiles() * D * 4 : 0;
  const Buf ws{need > 0 ? workspace : nullptr, need};
  if (clash({{y, n}, {s_out, st}, {ckpt, nck}, ws},
            {{q, n}, {k, n}, {v, n}, {g, ng}, {s0, st}}))
    return HYENA_ERR_INVALID_ARG;
  if (B * s.n_cb() * cuts_of(s).splits > kI32) return HYENA_ERR_UNSUPPORTED;
  hyena::host::DeviceInfo info;
  if (prepare_device(&info) != HYENA_OK) return HYENA_ERR_CUDA;
  sc::Params p = base_params(s, g, info);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.s0 = s0;
  p.s_out = s_out;
  p.ckpt = ckpt;
  p.y = y;
  p.fault = fault;
  if (wait_ns > 0) p.wait_ns = wait_ns;
  const int feed = choose_feed(s, {q, k, v}, {y}, g, 8, &p);
  return with_one_feed(feed, [&](auto f) {
    constexpr int kFeed = decltype(f)::value;
    if (dtype == HYENA_DTYPE_F32)
      return forward<sc::F32, kFeed>(s, p, workspace, info.sm_count, stream);
    return forward<sc::Bf16, kFeed>(s, p, workspace, info.sm_count, stream);
  });
}

}  // namespace

extern "C" {

int64_t hyena_scan_ckpt_tiles(int64_t L, int dtype) {
  const Shape s{1, L, 1, 1, dtype};
  if (check_shape(s) != HYENA_OK) return -HYENA_ERR_INVALID_ARG;
  return s.n_tiles();
}

int64_t hyena_scan_workspace_bytes(int64_t B, int64_t L, int64_t D, int d_g, int dtype) {
  const Shape s{B, L, D, d_g, dtype};
  if (check_shape(s) != HYENA_OK) return -HYENA_ERR_INVALID_ARG;
  return B == 0 || L == 0 ? 0 : agg_bytes(s);
}

int64_t hyena_scan_bwd_workspace_bytes(int64_t B, int64_t L, int64_t D, int d_g, int dtype,
                                       int have_ckpt) {
  const Shape s{B, L, D, d_g, dtype};
  if (check_shape(s) != HYENA_OK) return -HYENA_ERR_INVALID_ARG;
  if (B == 0 || L == 0) return 0;
  return agg_bytes(s) + dg_bytes(s) + (have_ckpt ? 0 : ckpt_bytes(s));
}

int hyena_scan_fwd(const void *q, const void *k, const void *v, const void *g, const float *s0,
                   void *y, float *s_out, float *ckpt, int64_t B, int64_t L, int64_t D, int d_g,
                   int dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  return scan_fwd(q, k, v, g, s0, y, s_out, ckpt, B, L, D, d_g, dtype, workspace, workspace_bytes,
                  0, 0, stream);
}

int hyena_testing_scan_fault(const void *q, const void *k, const void *v, const void *g, void *y,
                             float *s_out, int64_t B, int64_t L, int64_t D, int d_g, int dtype,
                             int fault, uint64_t wait_ns, cudaStream_t stream) {
  if (fault < 0 || fault > 1 || wait_ns < 1000000ull || wait_ns > hyena::kWaitTimeoutNs)
    return HYENA_ERR_INVALID_ARG;
  const Shape s{B, L, D, d_g, dtype};
  const int rc = check_shape(s);
  if (rc != HYENA_OK) return rc;
  if (B > 0 && L > 0 && cuts_of(s).cluster < 2) return HYENA_ERR_UNSUPPORTED;
  return scan_fwd(q, k, v, g, nullptr, y, s_out, nullptr, B, L, D, d_g, dtype, nullptr, 0, fault,
                  wait_ns, stream);
}

int hyena_scan_bwd(const void *q, const void *k, const void *v, const void *g, const float *s0,
                   const void *dy, const float *ds_out, const float *ckpt, void *dq, void *dk,
                   void *dv, void *dg, float *ds0, int64_t B, int64_t L, int64_t D, int d_g,
                   int dtype, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  const Shape s{B, L, D, d_g, dtype};
  int rc = check_shape(s);
  if (rc != HYENA_OK) return rc;
  if (misaligned(4, {s0, ds_out, ckpt, ds0})) return HYENA_ERR_MISALIGNED;
  if (B == 0) return HYENA_OK;
  const int64_t st = B * D * 4, n = s.numel() * s.es(), ng = B * L * s.G() * s.es();
  if (overlap(ds0, st, ds_out, st)) return HYENA_ERR_INVALID_ARG;
  if (L == 0) return copy_state(ds_out, ds0, B * D, stream);
  if (!q || !k || !v || !g || !dy || !dq || !dk || !dv || !dg) return HYENA_ERR_INVALID_ARG;
  if (misaligned(static_cast<uintptr_t>(s.es()), {q, k, v, g, dy, dq, dk, dv, dg}) ||
      !aligned(workspace, 16))
    return HYENA_ERR_MISALIGNED;
  const int64_t need = hyena_scan_bwd_workspace_bytes(B, L, D, d_g, dtype, ckpt != nullptr);
  if (need > 0 && (!workspace || static_cast<int64_t>(workspace_bytes) < need))
    return HYENA_ERR_INVALID_ARG;
  const int64_t nck = ckpt ? B * s.n_tiles() * D * 4 : 0;
  const Buf ws{need > 0 ? workspace : nullptr, need};
  if (clash({{dq, n}, {dk, n}, {dv, n}, {dg, ng}, {ds0, st}, ws},
            {{q, n}, {k, n}, {v, n}, {g, ng}, {dy, n}, {s0, st}, {ds_out, st}, {ckpt, nck}}))
    return HYENA_ERR_INVALID_ARG;
  if (B * s.n_cb() * cuts_of(s).splits > kI32) return HYENA_ERR_UNSUPPORTED;
  hyena::host::DeviceInfo info;
  if (prepare_device(&info) != HYENA_OK) return HYENA_ERR_CUDA;
  sc::Params p = base_params(s, g, info);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.dy = dy;
  p.s0 = s0;
  p.ds_out = ds_out;
  p.ckpt = const_cast<float *>(ckpt);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dg = dg;
  p.ds0 = ds0;
  const int raw = dtype == HYENA_DTYPE_F32 ? 0 : 2;
  const int feed = s.d_g == 1 ? choose_feed(s, {q, k, v, dy}, {dq, dk, dv, dg}, g, raw, &p)
                              : choose_feed(s, {q, k, v, dy}, {dq, dk, dv}, g, raw, &p);
  return with_one_feed(feed, [&](auto f) {
    constexpr int kFeed = decltype(f)::value;
    if constexpr (kFeed != sc::kTmaRaw)
      if (dtype == HYENA_DTYPE_F32)
        return backward<sc::F32, kFeed>(s, p, workspace, info.sm_count, stream);
    return backward<sc::Bf16, kFeed>(s, p, workspace, info.sm_count, stream);
  });
}

int hyena_scan_step(const void *q, const void *k, const void *v, const void *g, const float *s,
                    void *y, float *s_out, int64_t B, int64_t D, int d_g, int dtype,
                    cudaStream_t stream) {
  const Shape sh{B, 1, D, d_g, dtype};
  const int rc = check_shape(sh);
  if (rc != HYENA_OK) return rc;
  if (B == 0) return HYENA_OK;
  if (!q || !k || !v || !g || !s || !y || !s_out) return HYENA_ERR_INVALID_ARG;
  if (misaligned(static_cast<uintptr_t>(sh.es()), {q, k, v, g, y}) || misaligned(4, {s, s_out}))
    return HYENA_ERR_MISALIGNED;
  const int64_t st = B * D * 4, n = B * D * sh.es(), ng = B * sh.G() * sh.es();
  if ((s_out != s && overlap(s_out, st, s, st)) || overlap(y, n, s, st) ||
      clash({{y, n}, {s_out, st}}, {{q, n}, {k, n}, {v, n}, {g, ng}}))
    return HYENA_ERR_INVALID_ARG;
  const int vec = dtype == HYENA_DTYPE_F32 ? 4 : 8;
  const bool wide = D % vec == 0 && !misaligned(16, {q, k, v, y, s, s_out}) &&
                    (d_g > 1 || aligned(g, 16));
  const int64_t per = 128 * (wide ? vec : 1), blocks = (B * D + per - 1) / per;
  if (blocks > kI32) return HYENA_ERR_UNSUPPORTED;
  const auto go = [&](auto *type, auto vn) {
    using T = std::remove_pointer_t<decltype(type)>;
    return hyena::host::launch(sc::scan_step_kernel<T, decltype(vn)::value>,
                               dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream,
                               static_cast<const T *>(q), static_cast<const T *>(k),
                               static_cast<const T *>(v), static_cast<const T *>(g), s,
                               static_cast<T *>(y), s_out, B * D, static_cast<int>(D), d_g,
                               static_cast<int>(sh.G())) == cudaSuccess
               ? HYENA_OK
               : HYENA_ERR_CUDA;
  };
  if (dtype == HYENA_DTYPE_F32)
    return wide ? go(static_cast<float *>(nullptr), std::integral_constant<int, 4>())
                : go(static_cast<float *>(nullptr), std::integral_constant<int, 1>());
  return wide ? go(static_cast<__nv_bfloat16 *>(nullptr), std::integral_constant<int, 8>())
              : go(static_cast<__nv_bfloat16 *>(nullptr), std::integral_constant<int, 1>());
}

}  // extern "C"
