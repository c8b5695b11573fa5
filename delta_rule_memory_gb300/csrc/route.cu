// route.cu - visits sorted by partition and back.
//
// Token m of M makes k visits, visit m k + r to partition sel[m, r].  A stable counting sort gives each visit
// its place in the partition-sorted order; gather copies every token's row to its visits' places (the
// partitions' inputs), combine sums the rows at a token's places times its weights (the partitions' outputs).
// Either is the other's transpose: gather's gradient is combine without weights, combine's is a weighted gather
// and a dot product a visit.  Every sum is formed in a fixed order in fp32: no atomics.
//
// All of them move bytes and nothing else.  A warp has a token: its row is read (written) once and in whole
// lines, its places are k whole rows.
#include <climits>
#include <initializer_list>

#include <cuda_bf16.h>

#include "common.cuh"

namespace sdm {
namespace {

// ---------------------------------------------------------------------------
// The sort.  A block has kBlock visits, each of its warps a run of them, taken 32 at a time: lanes of one
// partition find one another with match_any, their order being the visits' own.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kRun = 128, kBlock = kSortWarps * kRun;
constexpr int kMaxParts = 1024;
// shared memory of the two kernels of N partitions, all of it dynamic: what decides whether a launch needs the raised
// limit is then the launch's own size
constexpr int count_smem(int N) { return kSortWarps * N * 4; }
constexpr int place_smem(int N) { return count_smem(N) + (2 * N + 1 + kSortWarps) * 4; }
constexpr int kSumHere = 8192;  // counts (blocks x N) up to which each block sums those before it by itself

struct SortArgs {
  const int32_t *sel;
  int64_t visits;
  int N, blocks;
  int32_t *order, *place, *offsets;
  int32_t *counts;  // [blocks][N]: visits of a block to a partition; then those of the blocks before it
  int32_t *err;
  int sum_here;
};

// the partitions of a warp's run of visits, N where there is none
struct Run {
  int p[kRun / 32];
};
__device__ __forceinline__ Run read_run(const SortArgs &a, int64_t first) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Run r;
#pragma unroll
  for (int o = 0; o < kRun / 32; ++o) {
    const int64_t i = first + w * kRun + 32 * o + lane;
    r.p[o] = i < a.visits ? a.sel[i] : -1;
  }
#pragma unroll
  for (int o = 0; o < kRun / 32; ++o) {
    if (r.p[o] >= a.N && a.err) atomicOr(a.err, SDM_DEVERR_INDEX_RANGE);
    if (r.p[o] < 0 || r.p[o] > a.N) r.p[o] = a.N;
  }
  return r;
}

// hist[warp][N]: each warp's visits to each partition
__device__ __forceinline__ void count_visits(const SortArgs &a, const Run &r, int *hist) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * a.N; i += kSortThreads) hist[i] = 0;
  __syncthreads();
#pragma unroll
  for (int o = 0; o < kRun / 32; ++o) {
    const uint32_t peers = __match_any_sync(kFull, r.p[o]);
    if (r.p[o] < a.N && (peers & ((1u << lane) - 1)) == 0) hist[w * a.N + r.p[o]] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) route_count(const SortArgs a) {
  extern __shared__ int hist[];
  count_visits(a, read_run(a, static_cast<int64_t>(blockIdx.x) * kBlock), hist);
  for (int p = threadIdx.x; p < a.N; p += kSortThreads) {
    int n = 0;
    for (int w = 0; w < kSortWarps; ++w) n += hist[w * a.N + p];
    a.counts[static_cast<int64_t>(blockIdx.x) * a.N + p] = n;
  }
}

// one warp a partition: its blocks' counts become those before each block; the total behind the last block
__global__ void __launch_bounds__(32) route_scan(const SortArgs a) {
  const int p = blockIdx.x, lane = threadIdx.x;
  int before = 0;
  for (int b = 0; b < a.blocks; b += 32) {
    const int64_t at = static_cast<int64_t>(b + lane) * a.N + p;
    const int n = b + lane < a.blocks ? a.counts[at] : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (b + lane < a.blocks) a.counts[at] = before + x - n;
    before += __shfl_sync(kFull, x, 31);
  }
  if (lane == 0) a.counts[static_cast<int64_t>(a.blocks) * a.N + p] = before;
}

// places.  One block alone counts for itself; with few counts in all a block sums those of the blocks before it
__global__ void __launch_bounds__(kSortThreads) route_place(const SortArgs a) {
  extern __shared__ int hist[];
  int *start = hist + kSortWarps * a.N, *ahead = start + a.N + 1, *sums = ahead + a.N;  // [N + 1], [N], [warps]
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kBlock;
  const Run run = read_run(a, first);
  count_visits(a, run, hist);
  // a partition's visits in the warps before, and its total
  for (int p = threadIdx.x; p < a.N; p += kSortThreads) {
    int n = 0;
    for (int i = 0; i < kSortWarps; ++i) {
      const int x = hist[i * a.N + p];
      hist[i * a.N + p] = n;
      n += x;
    }
    int before = 0;
    if (a.blocks > 1 && a.sum_here) {
      n = 0;
#pragma unroll 8
      for (int b = 0; b < a.blocks; ++b) {
        const int x = a.counts[b * a.N + p];
        n += x;
        before += b < static_cast<int>(blockIdx.x) ? x : 0;
      }
    } else if (a.blocks > 1) {
      n = a.counts[static_cast<int64_t>(a.blocks) * a.N + p];
      before = a.counts[static_cast<int64_t>(blockIdx.x) * a.N + p];
    }
    start[p] = n;
    ahead[p] = before;
  }
  __syncthreads();
  // totals to starts: kMaxParts / kSortThreads partitions a thread
  constexpr int each = kMaxParts / kSortThreads;
  int mine[each], n = 0;
#pragma unroll
  for (int e = 0; e < each; ++e) {
    const int p = threadIdx.x * each + e;
    mine[e] = n;
    n += p < a.N ? start[p] : 0;
  }
  int x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[w] = x;
  __syncthreads();
  int before = x - n, all = 0;
  for (int i = 0; i < kSortWarps; ++i) {
    if (i < w) before += sums[i];
    all += sums[i];
  }
#pragma unroll
  for (int e = 0; e < each; ++e) {
    const int p = threadIdx.x * each + e;
    if (p < a.N) start[p] = before + mine[e];
  }
  if (threadIdx.x == 0) start[a.N] = all;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int p = threadIdx.x; p <= a.N; p += kSortThreads) a.offsets[p] = start[p];
  for (int i = threadIdx.x; i < kSortWarps * a.N; i += kSortThreads) {
    const int p = i % a.N;
    hist[i] += start[p] + ahead[p];
  }
  __syncthreads();
#pragma unroll
  for (int o = 0; o < kRun / 32; ++o) {
    const int64_t i = first + w * kRun + 32 * o + lane;
    const int p = run.p[o];
    const uint32_t peers = __match_any_sync(kFull, p), below = peers & ((1u << lane) - 1);
    int at = -1;
    if (p < a.N) at = hist[w * a.N + p] + __popc(below);
    __syncwarp();
    if (p < a.N && below == 0) hist[w * a.N + p] += __popc(peers);
    __syncwarp();
    if (i < a.visits) {
      a.place[i] = at;
      if (at >= 0) a.order[at] = static_cast<int32_t>(i);
    }
  }
  for (int64_t j = all + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; j < a.visits;
       j += static_cast<int64_t>(gridDim.x) * kSortThreads)
    a.order[j] = -1;
}

// ---------------------------------------------------------------------------
// Rows there and back.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;

struct RowArgs {
  const void *x;      // gather: x [M, D]; backward: dy [M, D]
  const void *rows;   // combine, backward: [M k, D]
  void *out;          // gather, backward: [M k, D]; combine: y [M, D]
  int64_t ld;         // of x
  const int32_t *place, *offsets;
  const float *w;
  float *dw;
  int64_t M;
  int k, N, D;
};

// BYTES of a row as floats
template <typename T, int BYTES>
struct Piece {
  static constexpr int n = BYTES / sizeof(T);
  float v[n];
};
template <int BYTES>
struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

template <typename T, int BYTES>
__device__ __forceinline__ Piece<T, BYTES> unpack(const typename Raw<BYTES>::type &r) {
  Piece<T, BYTES> p;
  if constexpr (sizeof(T) == 4) {
    const float *f = reinterpret_cast<const float *>(&r);
#pragma unroll
    for (int i = 0; i < p.n; ++i) p.v[i] = f[i];
  } else {
    const uint16_t *f = reinterpret_cast<const uint16_t *>(&r);
#pragma unroll
    for (int i = 0; i < p.n; ++i) p.v[i] = bf16_to_f32(f[i]);
  }
  return p;
}
template <typename T, int BYTES>
__device__ __forceinline__ typename Raw<BYTES>::type pack(const Piece<T, BYTES> &p) {
  typename Raw<BYTES>::type r;
  if constexpr (sizeof(T) == 4) {
    float *f = reinterpret_cast<float *>(&r);
#pragma unroll
    for (int i = 0; i < p.n; ++i) f[i] = p.v[i];
  } else {
    uint16_t *f = reinterpret_cast<uint16_t *>(&r);
#pragma unroll
    for (int i = 0; i < p.n; ++i) f[i] = __bfloat16_as_ushort(__float2bfloat16_rn(p.v[i]));
  }
  return r;
}

// lane r's place of visit (m, r), -1 where it has none
__device__ __forceinline__ int place_of(const RowArgs &a, int64_t m, int lane) {
  const int at = lane < a.k ? a.place[m * a.k + lane] : -1;
  return at < a.M * a.k ? at : -1;
}

// rows of dropped visits, behind the last partition's: zeros
template <int BYTES>
__device__ __forceinline__ void clear_rest(const RowArgs &a, int pieces, int64_t warp, int64_t warps, int lane) {
  using R = typename Raw<BYTES>::type;
  for (int64_t j = max(a.offsets[a.N], 0) + warp; j < a.M * a.k; j += warps) {
    R *o = static_cast<R *>(a.out) + j * pieces;
    for (int c = lane; c < pieces; c += 32) o[c] = R{};
  }
}

// an item: a token and a stretch of 32 U pieces of its row
template <int BYTES>
constexpr int kStretch = BYTES == 16 ? 4 : 8;
struct Items {
  int64_t first, step, all;
  int each;  // stretches of a row
};
template <int U>
__device__ __forceinline__ Items items_of(const RowArgs &a, int pieces) {
  Items t;
  t.each = (pieces + 32 * U - 1) / (32 * U);
  t.first = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  t.step = static_cast<int64_t>(gridDim.x) * kRowWarps;
  t.all = a.M * t.each;
  return t;
}

template <int BYTES, int ES>
__global__ void __launch_bounds__(kRowThreads) route_gather_kernel(const RowArgs a) {
  using R = typename Raw<BYTES>::type;
  constexpr int U = kStretch<BYTES>;
  const int lane = threadIdx.x & 31, pieces = a.D / (BYTES / ES);
  const Items t = items_of<U>(a, pieces);
  for (int64_t it = t.first; it < t.all; it += t.step) {
    const int64_t m = it / t.each;
    const int c = static_cast<int>(it - m * t.each) * (32 * U) + lane;
    const int at = place_of(a, m, lane);
    const R *x = reinterpret_cast<const R *>(static_cast<const char *>(a.x) + m * a.ld * ES);
    R v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c + 32 * i < pieces) v[i] = x[c + 32 * i];
    for (int r = 0; r < a.k; ++r) {
      const int64_t j = __shfl_sync(kFull, at, r);
      if (j < 0) continue;
      R *o = static_cast<R *>(a.out) + j * pieces;
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + 32 * i < pieces) o[c + 32 * i] = v[i];
    }
  }
  clear_rest<BYTES>(a, pieces, t.first, t.step, lane);
}

// A row at a time, so that a thread needs few registers and an SM holds many warps, and reads that leave no
// trace in the caches (nothing is read twice): 16,384 x 4 rows of 3,840 bf16 in 101 us, 92% of the measured
// copy bandwidth, where four rows at a time took 133 and cached reads of two rows 182
template <typename T, int BYTES>
__global__ void __launch_bounds__(kRowThreads) route_combine_kernel(const RowArgs a) {
  using R = typename Raw<BYTES>::type;
  using P = Piece<T, BYTES>;
  constexpr int U = kStretch<BYTES>;
  const int lane = threadIdx.x & 31, pieces = a.D / P::n;
  const Items t = items_of<U>(a, pieces);
  for (int64_t it = t.first; it < t.all; it += t.step) {
    const int64_t m = it / t.each;
    const int c = static_cast<int>(it - m * t.each) * (32 * U) + lane;
    const int at = place_of(a, m, lane);
    const float wt = lane >= a.k ? 0.f : a.w ? a.w[m * a.k + lane] : 1.f;
    P sum[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int e = 0; e < P::n; ++e) sum[i].v[e] = 0.f;
    for (int r = 0; r < a.k; ++r) {
      const int64_t j = __shfl_sync(kFull, at, r);
      const float ww = __shfl_sync(kFull, wt, r);
      if (j < 0) continue;
      const R *x = static_cast<const R *>(a.rows) + j * pieces;
      R v[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + 32 * i < pieces) v[i] = __ldcs(x + c + 32 * i);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + 32 * i < pieces) {
          const P y = unpack<T, BYTES>(v[i]);
#pragma unroll
          for (int e = 0; e < P::n; ++e) sum[i].v[e] = fmaf(ww, y.v[e], sum[i].v[e]);
        }
    }
    R *y = static_cast<R *>(a.out) + m * pieces;
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (c + 32 * i < pieces) __stcs(y + c + 32 * i, pack<T, BYTES>(sum[i]));
  }
}

// V rows at a time: as many as a token has, up to four
template <typename T, int BYTES, int V>
__global__ void __launch_bounds__(kRowThreads) route_combine_back_kernel(const RowArgs a) {
  using R = typename Raw<BYTES>::type;
  using P = Piece<T, BYTES>;
  constexpr int U = 2;
  const int lane = threadIdx.x & 31, pieces = a.D / P::n;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5),
      warps = static_cast<int64_t>(gridDim.x) * kRowWarps;
  for (int64_t m = warp; m < a.M; m += warps) {
    const int at = place_of(a, m, lane);
    const float wt = lane < a.k ? a.w[m * a.k + lane] : 0.f;
    const R *dy = reinterpret_cast<const R *>(static_cast<const T *>(a.x) + m * a.ld);
    for (int r0 = 0; r0 < a.k; r0 += V) {
      int64_t j[V];
      float ww[V], dot[V];
#pragma unroll
      for (int r = 0; r < V; ++r) {
        j[r] = __shfl_sync(kFull, at, (r0 + r) & 31);
        ww[r] = __shfl_sync(kFull, wt, (r0 + r) & 31);
        if (r0 + r >= a.k) j[r] = -1;
        dot[r] = 0.f;
      }
      for (int c0 = 0; c0 < pieces; c0 += 32 * U) {
        const int c = c0 + lane;
        R d[U], v[V][U];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (c + 32 * i < pieces) d[i] = dy[c + 32 * i];
#pragma unroll
        for (int r = 0; r < V; ++r)
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (j[r] >= 0 && c + 32 * i < pieces)
              v[r][i] = (static_cast<const R *>(a.rows) + j[r] * pieces)[c + 32 * i];
#pragma unroll
        for (int r = 0; r < V; ++r)
#pragma unroll
          for (int i = 0; i < U; ++i)
            if (j[r] >= 0 && c + 32 * i < pieces) {
              const P x = unpack<T, BYTES>(v[r][i]);
              P y = unpack<T, BYTES>(d[i]);
#pragma unroll
              for (int e = 0; e < P::n; ++e) {
                dot[r] = fmaf(y.v[e], x.v[e], dot[r]);
                y.v[e] *= ww[r];
              }
              (static_cast<R *>(a.out) + j[r] * pieces)[c + 32 * i] = pack<T, BYTES>(y);
            }
      }
#pragma unroll
      for (int r = 0; r < V; ++r) {
#pragma unroll
        for (int o = 16; o; o >>= 1) dot[r] += __shfl_xor_sync(kFull, dot[r], o);
        if (lane == 0 && r0 + r < a.k) a.dw[m * a.k + r0 + r] = dot[r];
      }
    }
  }
  clear_rest<BYTES>(a, pieces, warp, warps, lane);
}

// the largest power of two up to 16 that divides every address and distance given
int piece_bytes(int es, int64_t D, int64_t ld, std::initializer_list<const void *> ptrs) {
  for (int n = 16; n > es; n /= 2) {
    bool ok = D * es % n == 0 && ld * es % n == 0;
    for (const void *p : ptrs) ok = ok && aligned(p, n);
    if (ok) return n;
  }
  return es;
}

unsigned row_grid(int64_t items) {
  // an item a warp; from 32 CTAs an SM on, warps take several
  const int64_t n = (items + kRowWarps - 1) / kRowWarps;
  return static_cast<unsigned>(n < 1 ? 1 : n > 152 * 32 ? 152 * 32 : n);
}

int check_rows(const char *what, int dtype, int64_t M, int k, int N, int D, int64_t ld) {
  if (M < 0 || k < 0 || N < 0 || D < 0) return set_error(SDM_ERR_INVALID_ARG, "%s: negative size", what);
  if (dtype != SDM_DTYPE_F32 && dtype != SDM_DTYPE_BF16)
    return set_error(SDM_ERR_UNSUPPORTED, "%s: unknown dtype", what);
  if (k > 32 || N > kMaxParts || M >= (1ll << 31) || M * k >= (1ll << 31) - kBlock || D >= (1 << 24))
    return set_error(SDM_ERR_SHAPE, "%s: need k <= 32, N <= %d, M k < 2^31 - 4096, D < 2^24", what, kMaxParts);
  if (ld < D || ld >= (1 << 27))
    return set_error(SDM_ERR_SHAPE, "%s: rows must be at least D and less than 2^27 elements apart", what);
  return SDM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" size_t route_sort_workspace_size(int64_t M, int k, int N) {
  if (M < 0 || k < 0 || N < 0 || k > 32 || N > kMaxParts || M >= (1ll << 31) || M * k >= (1ll << 31) - kBlock) return 0;
  const int64_t blocks = (M * k + kBlock - 1) / kBlock;
  return blocks <= 1 ? 0 : static_cast<size_t>(blocks + 1) * N * 4;
}

extern "C" int route_sort(const int32_t *sel, int64_t M, int k, int N, int32_t *order, int32_t *place, int32_t *offsets,
                          void *workspace, size_t workspace_bytes, int32_t *dev_err, void *stream) {
  const int rc = check_rows("route_sort", SDM_DTYPE_F32, M, k, N, 0, 0);
  if (rc != SDM_OK) return rc;
  if (!offsets || (M * k > 0 && (!sel || !order || !place)))
    return set_error(SDM_ERR_INVALID_ARG, "route_sort: null pointer");
  const size_t need = route_sort_workspace_size(M, k, N);
  if (need && (!workspace || workspace_bytes < need))
    return set_error(SDM_ERR_INVALID_ARG, "route_sort: workspace of %zu bytes needed", need);
  if (!aligned(sel, 4) || !aligned(order, 4) || !aligned(place, 4) || !aligned(offsets, 4) || !aligned(workspace, 4) ||
      !aligned(dev_err, 4))
    return set_error(SDM_ERR_ALIGN, "route_sort: a pointer is not aligned");
  SortArgs a{sel, M * k, N, static_cast<int>((M * k + kBlock - 1) / kBlock), order, place, offsets,
      static_cast<int32_t *>(workspace), dev_err, 0};
  if (a.blocks < 1) a.blocks = 1;
  a.sum_here = static_cast<int64_t>(a.blocks) * N <= kSumHere;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (place_smem(N) > 48 << 10)  // the limit is the kernel's, the same in every call
    for (const void *f : {reinterpret_cast<const void *>(route_count), reinterpret_cast<const void *>(route_place)}) {
      const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, place_smem(kMaxParts));
      if (e != cudaSuccess) return set_error(SDM_ERR_CUDA, "route_sort: %s", cudaGetErrorString(e));
    }
  if (a.blocks > 1 && N > 0) {
    route_count<<<a.blocks, kSortThreads, count_smem(N), st>>>(a);
    if (!a.sum_here) route_scan<<<N, 32, 0, st>>>(a);
  }
  route_place<<<a.blocks, kSortThreads, place_smem(N), st>>>(a);
  return check_launch("route_sort");
}

namespace {

// the kernel for an element type and a piece size: f(type tag, piece size tag)
template <int N>
struct Tag {
  static constexpr int value = N;
};
template <typename F>
void by_type(int dtype, int bytes, F f) {
  if (dtype == SDM_DTYPE_F32)
    bytes == 16 ? f(0.f, Tag<16>()) : bytes == 8 ? f(0.f, Tag<8>()) : f(0.f, Tag<4>());
  else
    bytes == 16  ? f(uint16_t(0), Tag<16>())
    : bytes == 8 ? f(uint16_t(0), Tag<8>())
    : bytes == 4 ? f(uint16_t(0), Tag<4>())
                 : f(uint16_t(0), Tag<2>());
}
// items of M rows in stretches of 32 u pieces
int64_t items(int64_t M, int D, int es, int bytes, int u) { return M * ((D / (bytes / es) + 32 * u - 1) / (32 * u)); }

}  // namespace

extern "C" int route_gather(const void *x, int64_t ld_x, int dtype, const int32_t *place, const int32_t *offsets,
                            int64_t M, int k, int N, int D, void *rows, void *stream) {
  const int rc = check_rows("route_gather", dtype, M, k, N, D, ld_x);
  if (rc != SDM_OK) return rc;
  if (M == 0 || k == 0 || D == 0) return SDM_OK;
  if (!x || !place || !offsets || !rows) return set_error(SDM_ERR_INVALID_ARG, "route_gather: null pointer");
  const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(rows, es) || !aligned(place, 4) || !aligned(offsets, 4))
    return set_error(SDM_ERR_ALIGN, "route_gather: a pointer is not aligned");
  RowArgs a{x, nullptr, rows, ld_x, place, offsets, nullptr, nullptr, M, k, N, D};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int bytes = piece_bytes(es, D, ld_x, {x, rows});
  by_type(dtype, bytes, [&](auto e, auto n) {
    const unsigned grid = row_grid(items(M, D, es, n.value, kStretch<n.value>));
    route_gather_kernel<n.value, sizeof e><<<grid, kRowThreads, 0, st>>>(a);
  });
  return check_launch("route_gather");
}

extern "C" int route_combine(const void *rows, int dtype, const int32_t *place, const float *w, int64_t M, int k, int D,
                             void *y, void *stream) {
  const int rc = check_rows("route_combine", dtype, M, k, 0, D, D);
  if (rc != SDM_OK) return rc;
  if (M == 0 || D == 0) return SDM_OK;
  if ((k > 0 && (!rows || !place)) || !y) return set_error(SDM_ERR_INVALID_ARG, "route_combine: null pointer");
  const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
  if (!aligned(rows, es) || !aligned(y, es) || !aligned(place, 4) || !aligned(w, 4))
    return set_error(SDM_ERR_ALIGN, "route_combine: a pointer is not aligned");
  RowArgs a{nullptr, rows, y, D, place, nullptr, w, nullptr, M, k, 0, D};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_type(dtype, piece_bytes(es, D, D, {rows, y}), [&](auto e, auto n) {
    const unsigned grid = row_grid(items(M, D, es, n.value, kStretch<n.value>));
    route_combine_kernel<decltype(e), n.value><<<grid, kRowThreads, 0, st>>>(a);
  });
  return check_launch("route_combine");
}

extern "C" int route_combine_backward(const void *dy, int64_t ld_dy, int dtype, const void *rows, const int32_t *place,
                                      const float *w, const int32_t *offsets, int64_t M, int k, int N, int D,
                                      void *drows, float *dw, void *stream) {
  const int rc = check_rows("route_combine_backward", dtype, M, k, N, D, ld_dy);
  if (rc != SDM_OK) return rc;
  if (M == 0 || k == 0) return SDM_OK;
  if (!place || !w || !offsets || !dw || (D > 0 && (!dy || !rows || !drows)))
    return set_error(SDM_ERR_INVALID_ARG, "route_combine_backward: null pointer");
  const int es = dtype == SDM_DTYPE_F32 ? 4 : 2;
  if (!aligned(dy, es) || !aligned(rows, es) || !aligned(drows, es) || !aligned(place, 4) || !aligned(w, 4) ||
      !aligned(offsets, 4) || !aligned(dw, 4))
    return set_error(SDM_ERR_ALIGN, "route_combine_backward: a pointer is not aligned");
  RowArgs a{dy, rows, drows, ld_dy, place, offsets, w, dw, M, k, N, D};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  by_type(dtype, piece_bytes(es, D, ld_dy, {dy, rows, drows}), [&](auto e, auto n) {
    if (k <= 2)
      route_combine_back_kernel<decltype(e), n.value, 2><<<row_grid(M), kRowThreads, 0, st>>>(a);
    else
      route_combine_back_kernel<decltype(e), n.value, 4><<<row_grid(M), kRowThreads, 0, st>>>(a);
  });
  return check_launch("route_combine_backward");
}
