// hyena_proj.cu -- host side of the projections (include/hyena_mixer.h): argument checks, the
// choice of tiles and k cuts, TMA descriptors and launches of the kernels in proj.cuh.
#include <algorithm>
#include <cstdint>
#include <limits>
#include <mutex>

#include "host_util.h"
#include "hyena_conv_testing.h"
#include "hyena_mixer.h"
#include "proj.cuh"

namespace {

namespace pj = hyena::proj;
using hyena::host::aligned;
using hyena::host::overlap;
using hyena::host::round_up;

constexpr int64_t kMaxDim = int64_t{1} << 30;
constexpr int64_t kMaxReduced = int64_t{1} << 24;  // a tile's sum ends well inside a wait's 2 s
constexpr int kSms = 148;
constexpr int kMaxSplits = 16;
// k-blocks that one bf16 accumulator takes at most.  It truncates at every addition, which on sums
// of one sign is a bias: the mean error of dw over 2^18 and 2^20 rows of positive values was 0.11
// and 0.67 percent (4096 x 4096 outputs; half a step of bf16 is 0.2 to 0.4).  Longer sums are cut,
// and the cuts added with rounding to nearest.
constexpr int64_t kMaxRun = 2048;

int64_t elem(int dtype) { return dtype == HYENA_DTYPE_F32 ? 4 : 2; }
int planes(int dtype) { return dtype == HYENA_DTYPE_F32 ? 3 : 1; }

// ------------------------------------------------------------------------------- plan
enum Shape { kPair256 = 0, kOne128 = 1, kOne64 = 2 };

struct TileShape {
  int m, n, workers;
  double block, block_f32, tail, epi;  // ns per k-block of 64 (of bf16, fp32 operands), outside the
                                       // k-blocks, and of a tile's epilogue
};
constexpr TileShape kShapes[] = {  // times measured on products of 16..8192 rows and columns
    {256, 256, kSms / 2, 340, 0, 5000, 3000},
    {128, 128, kSms, 230, 1150, 3200, 1500},
    {128, 64, kSms, 185, 950, 2600, 900}};

struct Plan {
  int shape, splits, kb, per;  // per: blocks per cut
  int64_t tiles_m, tiles_n, whole;
  bool join;  // the cuts of a tile are a cluster
};

// Clusters of so many CTAs, one per SM, that run at once (GPCs of 16 to 18 SMs; 16 clusters of 8
// took two waves).
constexpr int kMaxJoin = 8;
constexpr int kClusters[kMaxJoin + 1] = {0, 148, 66, 40, 32, 20, 16, 8, 8};

// The tile shape and the cuts along k with the least estimated time.  Persistent workers take the
// tiles in waves; those of an unfinished last wave (or, in a small problem, all) are cut so that
// the workers finish together, at the price of a second kernel over their partial sums; sums too
// long for one accumulator are cut in any case.  fp32 sums go on in registers, which hold no more
// than 128 x 128 outputs.
Plan find_plan(int64_t M, int64_t N, int64_t K, int dtype) {
  Plan best{};
  double best_ns = 0;
  const bool f32 = dtype == HYENA_DTYPE_F32;
  const int64_t total = (K + pj::kBK - 1) / pj::kBK;
  const int least = f32 ? 2 : 4;  // k-blocks worth a cut
  for (int s = f32 ? kOne128 : kPair256; s <= kOne64; ++s) {
    const TileShape &t = kShapes[s];
    const double block = f32 ? t.block_f32 : t.block;
    const int64_t tm = (M + t.m - 1) / t.m, tn = (N + t.n - 1) / t.n;
    const int64_t runs = f32 ? 1 : (total + kMaxRun - 1) / kMaxRun;  // cuts needed
    const int64_t whole = runs > 1 ? 0 : tm * tn / t.workers * t.workers, rest = tm * tn - whole;
    for (int64_t want = runs; want <= std::max<int64_t>(runs, rest ? kMaxSplits : 1); ++want) {
      const int64_t per = (total + want - 1) / want;
      const int splits = static_cast<int>((total + per - 1) / per);
      if (want > runs && (splits != want || per < least || rest * want > t.workers)) continue;
      // a tile's k-blocks run beside the epilogue of the one before it
      const int64_t waves = (rest * splits + t.workers - 1) / t.workers;
      double ns = static_cast<double>(whole / t.workers) * std::max(static_cast<double>(total) * block, t.epi) +
                  static_cast<double>(waves) *
                      std::max(static_cast<double>(per) * block, whole || waves > 1 ? t.epi : 0.0) +
                  t.tail;
      const bool join = splits > 1 && whole == 0 && s != kPair256 && splits <= kMaxJoin &&
                        rest <= kClusters[splits];
      if (join)
        ns += 1500;
      else if (splits > 1)  // the second kernel, and the partial sums' way to it and back
        ns += 3000 + static_cast<double>(rest * splits) * std::min<int64_t>(M, t.m) * t.n * 4 / 4500;
      if (best_ns == 0 || ns < best_ns) {
        best_ns = ns;
        best = Plan{s, splits, static_cast<int>(total), static_cast<int>(per), tm, tn, splits > 1 ? whole : tm * tn, join};
      }
    }
  }
  return best;
}

// The same, remembering the last few sizes a thread asked for (a call asks up to four times).
Plan plan_of(int64_t M, int64_t N, int64_t K, int dtype) {
  struct Entry {
    int64_t M, N, K;
    int dtype;
    Plan plan;
  };
  thread_local Entry seen[8] = {};
  thread_local unsigned next = 0;
  for (const Entry &e : seen)
    if (e.M == M && e.N == N && e.K == K && e.dtype == dtype) return e.plan;
  Entry &e = seen[next++ % 8];
  e = Entry{M, N, K, dtype, find_plan(M, N, K, dtype)};
  return e.plan;
}

// Whether a product's tiles and cuts cannot be counted in 32 bits.
bool too_many(int64_t M, int64_t N, int64_t K, int dtype) {
  const Plan p = plan_of(M, N, K, dtype);
  return p.tiles_m * p.tiles_n * p.splits > std::numeric_limits<int32_t>::max();
}

int64_t partial_bytes(int64_t M, int64_t N, int64_t K, int dtype) {
  const Plan p = plan_of(M, N, K, dtype);
  const int64_t cut = p.join ? 0 : (p.tiles_m * p.tiles_n - p.whole) * p.splits;
  return cut * kShapes[p.shape].m * kShapes[p.shape].n * 4;  // a multiple of 256
}

// An operand [rows][cols] in memory: `ptr` with rows of `ld` elements, as bf16 planes.
struct Operand {
  const void *ptr;
  int64_t rows, cols, ld;
};

bool needs_pack(int64_t cols, int dtype) { return dtype == HYENA_DTYPE_F32 || cols % 8 != 0; }
int64_t pack_bytes(int64_t rows, int64_t cols, int dtype) {
  return round_up(planes(dtype) * rows * round_up(cols, 8) * 2, 256);
}

int encode(CUtensorMap *m, const Operand &o, int n_planes, int box_rows) {
  hyena::host::EncodeTiledFn enc = hyena::host::encode_tiled();
  if (!enc) return HYENA_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(n_planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2,
                                 static_cast<cuuint64_t>(o.rows * o.ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(o.ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

// An output (or residual) [M, N] of bf16 as the epilogue's chunks of 32 x 32.
int encode_out(CUtensorMap *m, const void *ptr, int64_t M, int64_t N) {
  hyena::host::EncodeTiledFn enc = hyena::host::encode_tiled();
  if (!enc) return HYENA_ERR_CUDA;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(N) * 2, static_cast<cuuint64_t>(M * N) * 2};
  const cuuint32_t box[3] = {pj::kChunk, 32, 1}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

// ------------------------------------------------------------------------------- launches
struct Device {
  hyena::host::DeviceInfo info;
  int pairs;  // resident pairs of CTAs
};

template <typename T, int kCG, int kBN, bool kAMn, bool kBMn, bool kJoin>
cudaError_t allow(int *resident) {
  using L = pj::Tile<kCG, kBN>;
  auto *fn = pj::proj_kernel<T, kCG, kBN, kAMn, kBMn, kJoin>;
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e == cudaSuccess && kCG == 2 && resident) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kSms);
    cfg.blockDim = dim3(pj::kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(resident, fn, &cfg);
  }
  return e;
}
template <typename T, bool kAMn, bool kBMn>
cudaError_t allow_all(int *resident) {
  cudaError_t e = cudaSuccess;
  if constexpr (sizeof(T) == 2) e = allow<T, 2, 256, kAMn, kBMn, false>(resident);
  if (e == cudaSuccess) e = allow<T, 1, 128, kAMn, kBMn, false>(nullptr);
  if (e == cudaSuccess) e = allow<T, 1, 64, kAMn, kBMn, false>(nullptr);
  if (e == cudaSuccess) e = allow<T, 1, 128, kAMn, kBMn, true>(nullptr);
  if (e == cudaSuccess) e = allow<T, 1, 64, kAMn, kBMn, true>(nullptr);
  return e;
}

int prepare_device(Device *d) {
  if (hyena::host::device_info(&d->info) != HYENA_OK) return HYENA_ERR_CUDA;
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static cudaError_t err[kMaxDevices];
  static int pairs[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return HYENA_ERR_CUDA;
  std::call_once(once[dev], [dev]() {
    int r = 0;
    cudaError_t e = allow_all<float, false, false>(nullptr);
    if (e == cudaSuccess) e = allow_all<float, false, true>(nullptr);
    if (e == cudaSuccess) e = allow_all<float, true, true>(nullptr);
    if (e == cudaSuccess) e = allow_all<__nv_bfloat16, false, false>(&r);
    if (e == cudaSuccess) e = allow_all<__nv_bfloat16, false, true>(nullptr);
    if (e == cudaSuccess) e = allow_all<__nv_bfloat16, true, true>(nullptr);
    err[dev] = e;
    pairs[dev] = std::max(1, r);
  });
  d->pairs = pairs[dev];
  return err[dev] == cudaSuccess ? HYENA_OK : HYENA_ERR_CUDA;
}

template <typename T, int kCG, int kBN, bool kAMn, bool kBMn, bool kJoin = false>
cudaError_t launch_shape(const CUtensorMap (&m)[5], const pj::Params &p, const Device &d,
                         cudaStream_t stream) {
  using L = pj::Tile<kCG, kBN>;
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const int64_t works = p.whole + (tiles - p.whole) * p.splits;
  const int64_t workers =
      kJoin ? works : std::min<int64_t>(works, kCG == 2 ? d.pairs : d.info.sm_count);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(kJoin ? p.splits : 2), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(workers * kCG));
  cfg.blockDim = dim3(pj::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = kCG == 2 || kJoin ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, pj::proj_kernel<T, kCG, kBN, kAMn, kBMn, kJoin>, m[0], m[1], m[2], m[3],
                            m[4], p);
}

// C = A B^T with its epilogue.  p: outputs, epilogue and status; K: the reduced dimension.  a, b:
// operands as they lie (kAMn / kBMn: [k][m] / [k][n]).
template <typename T, bool kAMn, bool kBMn>
int product(const Operand &a, const Operand &b, int64_t K, pj::Params p, int dtype, float *partial,
            const Device &d, cudaStream_t stream) {
  const Plan pl = plan_of(p.M, p.N, K, dtype);
  p.kb = pl.kb;
  p.tiles_m = static_cast<int>(pl.tiles_m);
  p.tiles_n = static_cast<int>(pl.tiles_n);
  p.whole = static_cast<int>(pl.whole);
  p.splits = pl.splits;
  p.kb_per_split = pl.per;
  p.group_m = pl.shape == kPair256 ? 8 : 16;
  if (p.wait_ns == 0) p.wait_ns = hyena::kWaitTimeoutNs;
  p.partial = partial;
  const int64_t per16 = 16 / elem(dtype);
  p.vec = p.N % per16 == 0 && aligned(p.y, 16) && aligned(p.z, 16) && aligned(p.residual, 16);
  p.bias_vec = aligned(p.bias, 16);
  p.tma = sizeof(T) == 2 && p.vec && p.whole > 0 && !(p.z && p.residual);
  CUtensorMap m[5] = {};  // A, B, y, z, residual
  const int b_rows = pl.shape == kOne64 ? 64 : 128;
  if (encode(&m[0], a, planes(dtype), kAMn ? 64 : pj::kRows) ||
      encode(&m[1], b, planes(dtype), kBMn ? 64 : b_rows) ||
      (p.tma && encode_out(&m[2], p.y, p.M, p.N)) ||
      (p.tma && p.z && encode_out(&m[3], p.z, p.M, p.N)) ||
      (p.tma && p.residual && encode_out(&m[4], p.residual, p.M, p.N)))
    return HYENA_ERR_CUDA;
  cudaError_t e;
  switch (pl.shape) {
    case kPair256:
      if constexpr (sizeof(T) == 2) {
        e = launch_shape<T, 2, 256, kAMn, kBMn>(m, p, d, stream);
        break;
      } else {
        return HYENA_ERR_UNSUPPORTED;  // not planned for fp32
      }
    case kOne128:
      e = pl.join ? launch_shape<T, 1, 128, kAMn, kBMn, true>(m, p, d, stream)
                  : launch_shape<T, 1, 128, kAMn, kBMn>(m, p, d, stream);
      break;
    default:
      e = pl.join ? launch_shape<T, 1, 64, kAMn, kBMn, true>(m, p, d, stream)
                  : launch_shape<T, 1, 64, kAMn, kBMn>(m, p, d, stream);
  }
  if (e != cudaSuccess) return HYENA_ERR_CUDA;
  if (p.splits == 1 || pl.join) return HYENA_OK;
  const TileShape &t = kShapes[pl.shape];
  const int64_t rest = pl.tiles_m * pl.tiles_n - pl.whole;
  const int64_t quads = std::min<int64_t>(t.m, p.M) * (t.n / 4);
  const int64_t want = std::max<int64_t>(1, 8 * d.info.sm_count / rest);
  const dim3 grid(static_cast<unsigned>(std::min((quads + 255) / 256, want)),
                  static_cast<unsigned>(std::min<int64_t>(rest, 65535)));
  const auto join = [&](auto *kernel) {
    return hyena::host::launch(kernel, grid, dim3(256), 0, stream, p);
  };
  switch (pl.shape) {
    case kPair256:
      if constexpr (sizeof(T) == 2) e = join(pj::proj_join_kernel<T, 256, 256>);
      break;
    case kOne128: e = join(pj::proj_join_kernel<T, 128, 128>); break;
    default: e = join(pj::proj_join_kernel<T, 128, 64>);
  }
  return e == cudaSuccess ? HYENA_OK : HYENA_ERR_CUDA;
}

// Up to two inputs of one row length as operands: themselves, or (`at` advances) bf16 planes in
// the workspace.  Rows 0: none.
template <typename T>
int operands(Operand *a, const void *pa, int64_t ra, Operand *b, const void *pb, int64_t rb,
             int64_t cols, int dtype, uint8_t *&at, const Device &d, cudaStream_t stream) {
  *a = Operand{pa, ra, cols, cols};
  *b = Operand{pb, rb, cols, cols};
  if (!needs_pack(cols, dtype)) return HYENA_OK;
  const int64_t ld = round_up(cols, 8), n = (ra + rb) * (ld / 8);
  const auto place = [&](Operand *o, const void *ptr, int64_t rows) {
    const pj::Pack<T> p{static_cast<const T *>(ptr), reinterpret_cast<__nv_bfloat16 *>(at), rows};
    *o = Operand{at, rows, cols, ld};
    at += pack_bytes(rows, cols, dtype);
    return p;
  };
  const pj::Pack<T> ka = place(a, pa, ra), kb = place(b, pb, rb);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 16 * d.info.sm_count));
  return hyena::host::launch(pj::proj_pack_kernel<T>, dim3(grid), dim3(256), 0, stream, ka, kb,
                             static_cast<int>(cols), static_cast<int>(ld)) == cudaSuccess
             ? HYENA_OK
             : HYENA_ERR_CUDA;
}

int check_shape(int64_t M, int64_t N, int64_t K, int dtype) {
  if (dtype != HYENA_DTYPE_BF16 && dtype != HYENA_DTYPE_F32) return HYENA_ERR_INVALID_ARG;
  if (M < 0 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxReduced)
    return HYENA_ERR_INVALID_ARG;
  return HYENA_OK;
}

struct Buf {
  const void *p;
  int64_t bytes;
};
bool clash(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf *o = outs.begin(); o != outs.end(); ++o) {
    for (const Buf &i : ins)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return true;
    for (const Buf *q = o + 1; q != outs.end(); ++q)
      if (overlap(o->p, o->bytes, q->p, q->bytes)) return true;
  }
  return false;
}

template <typename T>
int forward(const void *x, const void *w, const pj::Params &p, int64_t K, int dtype, uint8_t *ws,
            const Device &d, cudaStream_t stream) {
  Operand a, b;
  const int rc = operands<T>(&a, x, p.M, &b, w, p.N, K, dtype, ws, d, stream);
  if (rc != HYENA_OK) return rc;
  return product<T, false, false>(a, b, K, p, dtype, reinterpret_cast<float *>(ws), d, stream);
}

// Rows whose sum a CTA of the dz kernel leaves: all of them where they are few, which spares the
// kernel that adds up the blocks.
int64_t db_rows(int64_t M) { return M <= 512 ? 512 : 128; }
int64_t db_blocks(int64_t M) { return (M + db_rows(M) - 1) / db_rows(M); }

template <typename T, int kAct>
cudaError_t launch_dz(const void *dy, const void *z, __nv_bfloat16 *dz, float *part, int64_t M,
                      int64_t N, int64_t ld, int vec, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((ld + pj::kDbCols - 1) / pj::kDbCols),
                  static_cast<unsigned>(db_blocks(M)));
  return hyena::host::launch(pj::proj_dz_kernel<T, kAct>, grid, dim3(256), 0, stream,
                             static_cast<const T *>(dy), static_cast<const T *>(z), dz, part, M,
                             static_cast<int>(N), static_cast<int>(ld), vec,
                             static_cast<int>(db_rows(M)));
}

bool needs_dz(int64_t N, int act, int dtype) {
  return act != HYENA_ACT_NONE || needs_pack(N, dtype);
}

template <typename T>
int backward(const void *x, const void *w, const void *z, const void *dy, const void *dx_add,
             void *dx, void *dw, float *db, int64_t M, int64_t N, int64_t K, int act, int dtype,
             uint8_t *ws, const Device &d, cudaStream_t stream) {
  Operand dzo{dy, M, N, N};
  const bool make_dz = needs_dz(N, act, dtype) && (dx || dw);
  if (make_dz || db) {
    const int64_t ld = round_up(N, 8);
    __nv_bfloat16 *dz = nullptr;
    if (make_dz) {
      dz = reinterpret_cast<__nv_bfloat16 *>(ws);
      dzo = Operand{ws, M, N, ld};
      ws += pack_bytes(M, N, dtype);
    }
    float *part = nullptr;
    if (db) {
      part = db_blocks(M) > 1 ? reinterpret_cast<float *>(ws) : db;
      ws += round_up(db_blocks(M) * N * 4, 256);
    }
    const int vec = N % (16 / elem(dtype)) == 0 ? 1 : 0;
    cudaError_t e;
    switch (act) {
      case HYENA_ACT_GELU: e = launch_dz<T, pj::kGelu>(dy, z, dz, part, M, N, ld, vec, stream); break;
      case HYENA_ACT_SILU: e = launch_dz<T, pj::kSilu>(dy, z, dz, part, M, N, ld, vec, stream); break;
      case HYENA_ACT_SIGMOID:
        e = launch_dz<T, pj::kSigmoid>(dy, z, dz, part, M, N, ld, vec, stream);
        break;
      case HYENA_ACT_LOGSIGMOID:
        e = launch_dz<T, pj::kLogSigmoid>(dy, z, dz, part, M, N, ld, vec, stream);
        break;
      default: e = launch_dz<T, pj::kNone>(dy, z, dz, part, M, N, ld, vec, stream);
    }
    if (e == cudaSuccess && db && db_blocks(M) > 1)
      e = hyena::host::launch(pj::proj_db_kernel, dim3(static_cast<unsigned>((N + 31) / 32)),
                              dim3(256), 0, stream, static_cast<const float *>(part), db,
                              static_cast<int>(db_blocks(M)), static_cast<int>(N));
    if (e != cudaSuccess) return HYENA_ERR_CUDA;
  }
  pj::Params p{};
  p.status = d.info.status;
  p.act = pj::kNone;
  int rc = HYENA_OK;
  Operand xo, wo;
  if (dx || dw) {
    rc = operands<T>(&xo, x, dw ? M : 0, &wo, w, dx ? N : 0, K, dtype, ws, d, stream);
    if (rc != HYENA_OK) return rc;
  }
  if (dx) {  // [M, K] = dz [M, N] w [N, K]
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(K);
    p.residual = dx_add;
    p.y = dx;
    rc = product<T, false, true>(dzo, wo, N, p, dtype, reinterpret_cast<float *>(ws), d, stream);
    if (rc != HYENA_OK) return rc;
  }
  if (dw) {  // [N, K] = dz^T [N, M] x [M, K]
    p.M = static_cast<int>(N);
    p.N = static_cast<int>(K);
    p.residual = nullptr;
    p.y = dw;
    rc = product<T, true, true>(dzo, xo, M, p, dtype, reinterpret_cast<float *>(ws), d, stream);
  }
  return rc;
}

bool misaligned16(std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs)
    if (!aligned(p, 16)) return true;
  return false;
}

// hyena_proj_fwd with the test settings of hyena_testing_proj_fault (0, 0 in the product path).
int proj_fwd(const void *x, const void *w, const float *bias, const void *residual, void *y,
             void *z, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace,
             size_t workspace_bytes, int fault, uint64_t wait_ns, cudaStream_t stream) {
  const int rc = check_shape(M, N, K, dtype);
  if (rc != HYENA_OK) return rc;
  if (act < HYENA_ACT_NONE || act > HYENA_ACT_LOGSIGMOID) return HYENA_ERR_INVALID_ARG;
  if (M == 0) return HYENA_OK;
  if (!x || !w || !y) return HYENA_ERR_INVALID_ARG;
  if (misaligned16({x, w, residual, y, z}) || !aligned(bias, 4) || !aligned(workspace, 256))
    return HYENA_ERR_MISALIGNED;
  const int64_t need = hyena_proj_workspace_bytes(M, N, K, dtype), es = elem(dtype);
  if (need < 0) return static_cast<int>(-need);
  if (need > 0 && (!workspace || static_cast<int64_t>(workspace_bytes) < need))
    return HYENA_ERR_INVALID_ARG;
  const int64_t nx = M * K * es, nw = N * K * es, ny = M * N * es;
  const Buf ws{need > 0 ? workspace : nullptr, need};
  if (clash({{y, ny}, {z, ny}, ws}, {{x, nx}, {w, nw}, {bias, N * 4}}) ||
      clash({{z, ny}, ws}, {{residual, ny}}) || (residual != y && overlap(residual, ny, y, ny)))
    return HYENA_ERR_INVALID_ARG;
  Device d;
  if (prepare_device(&d) != HYENA_OK) return HYENA_ERR_CUDA;
  pj::Params p{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.bias = bias;
  p.residual = residual;
  p.y = y;
  p.z = z;
  p.act = act;
  p.status = d.info.status;
  p.fault = fault;
  p.wait_ns = wait_ns;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  return dtype == HYENA_DTYPE_F32 ? forward<float>(x, w, p, K, dtype, at, d, stream)
                                  : forward<__nv_bfloat16>(x, w, p, K, dtype, at, d, stream);
}

}  // namespace

extern "C" {

int64_t hyena_proj_workspace_bytes(int64_t M, int64_t N, int64_t K, int dtype) {
  if (check_shape(M, N, K, dtype) != HYENA_OK) return -HYENA_ERR_INVALID_ARG;
  if (M == 0) return 0;
  if (too_many(M, N, K, dtype)) return -HYENA_ERR_UNSUPPORTED;
  int64_t n = partial_bytes(M, N, K, dtype);
  if (needs_pack(K, dtype)) n += pack_bytes(M, K, dtype) + pack_bytes(N, K, dtype);
  return n;
}

int64_t hyena_proj_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int act, int dtype) {
  if (check_shape(M, N, K, dtype) != HYENA_OK || act < HYENA_ACT_NONE || act > HYENA_ACT_LOGSIGMOID)
    return -HYENA_ERR_INVALID_ARG;
  if (M == 0) return 0;
  if (db_blocks(M) > 65535 || N > kMaxReduced || too_many(M, K, N, dtype) ||
      too_many(N, K, M, dtype))
    return -HYENA_ERR_UNSUPPORTED;
  int64_t n = round_up(db_blocks(M) * N * 4, 256);
  if (needs_dz(N, act, dtype)) n += pack_bytes(M, N, dtype);
  if (needs_pack(K, dtype)) n += pack_bytes(M, K, dtype) + pack_bytes(N, K, dtype);
  // the two products run one after the other and share the room for partial sums
  return n + std::max(partial_bytes(M, K, N, dtype), partial_bytes(N, K, M, dtype));
}

int hyena_proj_fwd(const void *x, const void *w, const float *bias, const void *residual, void *y,
                   void *z, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace,
                   size_t workspace_bytes, cudaStream_t stream) {
  return proj_fwd(x, w, bias, residual, y, z, M, N, K, act, dtype, workspace, workspace_bytes,
                  pj::kNoFault, 0, stream);
}

int hyena_testing_proj_fault(const void *x, const void *w, const void *residual, void *y,
                             int64_t M, int64_t N, int64_t K, int fault, uint64_t wait_ns,
                             cudaStream_t stream) {
  if (fault < pj::kNoFault || fault > pj::kStagesEnd || wait_ns < 1000000ull ||
      wait_ns > hyena::kWaitTimeoutNs)
    return HYENA_ERR_INVALID_ARG;
  if (N % 8 != 0 || hyena_proj_workspace_bytes(M, N, K, HYENA_DTYPE_BF16) != 0)
    return HYENA_ERR_UNSUPPORTED;
  return proj_fwd(x, w, nullptr, residual, y, nullptr, M, N, K, HYENA_ACT_NONE, HYENA_DTYPE_BF16,
                  nullptr, 0, fault, wait_ns, stream);
}

int hyena_proj_bwd(const void *x, const void *w, const void *z, const void *dy,
                   const void *dx_add, void *dx, void *dw, float *db, int64_t M, int64_t N,
                   int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
  const int rc = check_shape(M, N, K, dtype);
  if (rc != HYENA_OK) return rc;
  if (act < HYENA_ACT_NONE || act > HYENA_ACT_LOGSIGMOID) return HYENA_ERR_INVALID_ARG;
  if (misaligned16({x, w, z, dy, dx_add, dx, dw}) || !aligned(db, 4) || !aligned(workspace, 256))
    return HYENA_ERR_MISALIGNED;
  const int64_t es = elem(dtype), nx = M * K * es, nw = N * K * es, ny = M * N * es;
  if (M == 0) {
    if ((dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(nw), stream) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 4, stream) != cudaSuccess))
      return HYENA_ERR_CUDA;
    return HYENA_OK;
  }
  if (!dy || (dx && !w) || (dw && !x) || (act != HYENA_ACT_NONE && !z)) return HYENA_ERR_INVALID_ARG;
  const int64_t need = hyena_proj_bwd_workspace_bytes(M, N, K, act, dtype);
  if (need < 0) return static_cast<int>(-need);
  if (!workspace || static_cast<int64_t>(workspace_bytes) < need) return HYENA_ERR_INVALID_ARG;
  if (clash({{dx, nx}, {dw, nw}, {db, N * 4}, {workspace, need}},
            {{x, nx}, {w, nw}, {z, ny}, {dy, ny}}) ||
      clash({{dw, nw}, {db, N * 4}, {workspace, need}}, {{dx_add, nx}}) ||
      (dx_add != dx && overlap(dx_add, nx, dx, nx)))
    return HYENA_ERR_INVALID_ARG;
  Device d;
  if (prepare_device(&d) != HYENA_OK) return HYENA_ERR_CUDA;
  uint8_t *at = static_cast<uint8_t *>(workspace);
  return dtype == HYENA_DTYPE_F32
             ? backward<float>(x, w, z, dy, dx_add, dx, dw, db, M, N, K, act, dtype, at, d, stream)
             : backward<__nv_bfloat16>(x, w, z, dy, dx_add, dx, dw, db, M, N, K, act, dtype, at, d,
                                       stream);
}

}  // extern "C"
