// route.cu -- tokens sorted by expert and back: hq_moe_sort (a stable counting
// sort of the (token, slot) pairs), hq_moe_gather and hq_moe_combine, and
// their gradients.
//
// All four row movers go by pos[t][j], the row of pair (t, j), so a token's
// sum runs over its slots in ascending order in fp32 (no atomics: results do
// not depend on the order of anything).  Bound: HBM; every row is read and
// written once, 16 bytes a thread where width and pointers allow.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "hq_common.cuh"
#include "hq_internal.h"
#include "hq_io.cuh"
#include "hq_launch.cuh"
#include "route.cuh"

namespace hq {
namespace route {
namespace {

constexpr int kSortThreads = 512;
constexpr int kOneTile = 2048;      // pairs that one block sorts alone
constexpr int kMinTile = 1024;      // pairs per block of more
constexpr int kMaxTiles = 64;       // blocks of one sort: each reads all blocks' histograms
constexpr int kMaxExperts = 16384;
constexpr long kMaxPairs = 1l << 23;

// Warps that count a tile side by side: each has its own histogram in shared
// memory, at most 128 KiB in all.
__host__ __device__ constexpr int sort_warps(int E) {
  return E <= 2048 ? 16 : 32768 / E;
}

struct SortArgs {
  const int32_t* ids;
  int P, E, align, tiles, tile;  // pairs, ..., blocks and pairs per block
  int bits;                      // of 0 .. E (E: no expert)
  int32_t* pos;
  int32_t* offsets;  // [E + 1]
  int32_t* counts;   // [E]
  int32_t* hist;     // [tiles][E] (more than one tile)
};

// The pairs of warp w's share of tile b, 32 at a time; four loads in flight.
template <typename F>
__device__ __forceinline__ void each_pair(const SortArgs& a, int b, int w, int W, F&& f) {
  const int lane = threadIdx.x & 31;
  const int t0 = b * a.tile, t1 = min(a.P, t0 + a.tile);
  const int per = ((t1 - t0 + W - 1) / W + 31) / 32 * 32;
  const int p1 = min(t1, t0 + (w + 1) * per);
  for (int p = t0 + w * per; p < p1; p += 128) {
    int id[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) id[u] = p + 32 * u + lane < p1 ? __ldg(a.ids + p + 32 * u + lane) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = p + 32 * u + lane;
      if (p + 32 * u < p1) f(i, i < p1, id[u], static_cast<uint32_t>(id[u]) < static_cast<uint32_t>(a.E));
    }
  }
}

// The lanes that hold the same id, by a ballot per bit of the id (fewer cycles
// than match.any over many different ids: 4084 pairs in one block 10.0 us with
// it, 7.9 us so).
__device__ __forceinline__ uint32_t same_id(int id, int bits) {
  uint32_t m = ~0u;
  for (int b = 0; b < bits; ++b) {
    const bool one = id >> b & 1;
    const uint32_t v = __ballot_sync(~0u, one);
    m &= one ? v : ~v;
  }
  return m;
}

__device__ __forceinline__ void count_tile(const SortArgs& a, int b, int32_t* h) {
  const int W = sort_warps(a.E), w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < W * a.E; i += kSortThreads) h[i] = 0;
  __syncthreads();
  if (w < W) {
    int32_t* mine = h + w * a.E;
    each_pair(a, b, w, W, [&](int, bool, int id, bool ok) {
      const uint32_t same = same_id(ok ? id : a.E, a.bits);
      if (ok && (same & ((1u << lane) - 1)) == 0) mine[id] += __popc(same);
      __syncwarp();
    });
  }
  __syncthreads();
}

// Histogram of every tile (only launched for more than one).
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortArgs a) {
  extern __shared__ int32_t h[];
  pdl_wait();
  pdl_launch_dependents();
  count_tile(a, blockIdx.x, h);
  const int W = sort_warps(a.E);
  for (int e = threadIdx.x; e < a.E; e += kSortThreads) {
    int n = 0;
#pragma unroll 8
    for (int w = 0; w < W; ++w) n += h[w * a.E + e];
    a.hist[static_cast<size_t>(blockIdx.x) * a.E + e] = n;
  }
}

// Rows of one tile's pairs: the experts' aligned segment starts (a scan over
// the counts, done by every block), plus the pairs of the same expert in
// earlier tiles, in earlier warps' shares and earlier in this share.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const SortArgs a) {
  extern __shared__ int32_t h[];
  __shared__ int32_t warp_sum[kSortThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int W = sort_warps(a.E), w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count_tile(a, blockIdx.x, h);
  int32_t carry = 0;  // aligned rows of the experts before e0
  for (int e0 = 0; e0 < a.E; e0 += kSortThreads) {
    const int e = e0 + threadIdx.x;
    int total = 0, before = 0;
    if (e < a.E) {
      if (a.tiles == 1) {
#pragma unroll 8
        for (int i = 0; i < W; ++i) total += h[i * a.E + e];
      } else {
#pragma unroll 8
        for (int b = 0; b < a.tiles; ++b) {
          const int n = __ldcg(a.hist + static_cast<size_t>(b) * a.E + e);
          before += b < static_cast<int>(blockIdx.x) ? n : 0;
          total += n;
        }
      }
    }
    const int rows = (total + a.align - 1) / a.align * a.align;
    int scan = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[w] = scan;
    __syncthreads();
    if (w == 0) {
      int s = lane < kSortThreads / 32 ? warp_sum[lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += v;
      }
      if (lane < kSortThreads / 32) warp_sum[lane] = s;
    }
    __syncthreads();
    const int start = carry + (w > 0 ? warp_sum[w - 1] : 0) + scan - rows;
    carry += warp_sum[kSortThreads / 32 - 1];
    if (e < a.E) {
      if (blockIdx.x == 0) {
        a.offsets[e] = start;
        a.counts[e] = total;
        if (e == a.E - 1) a.offsets[a.E] = start + rows;
      }
      int run = start + before;
#pragma unroll 8
      for (int i = 0; i < W; ++i) {
        const int n = h[i * a.E + e];
        h[i * a.E + e] = run;
        run += n;
      }
    }
    __syncthreads();
  }
  if (w < W) {
    int32_t* mine = h + w * a.E;
    each_pair(a, blockIdx.x, w, W, [&](int i, bool in, int id, bool ok) {
      const uint32_t same = same_id(ok ? id : a.E, a.bits);
      const uint32_t below = same & ((1u << lane) - 1);
      const int row = ok ? mine[id] + __popc(below) : -1;
      __syncwarp();
      if (ok && below == 0) mine[id] += __popc(same);
      __syncwarp();
      if (in) a.pos[i] = row;
    });
  }
}

// 16 bytes of T, or one value where rows are not made of whole vectors.
template <typename T, bool VEC>
struct Piece {
  static constexpr int N = VEC ? 16 / sizeof(T) : 1;
  float v[N];
  using Raw = typename std::conditional<VEC, uint4, T>::type;
  static __device__ __forceinline__ Raw raw(const T* p) {
    if constexpr (VEC) return __ldg(reinterpret_cast<const uint4*>(p));
    else return __ldg(p);
  }
  __device__ __forceinline__ void unpack(const Raw& u) {
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32<T>(t[i]);
  }
  __device__ __forceinline__ void load(const T* p) { unpack(raw(p)); }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC) {
      uint4 u;
      T* t = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      *p = from_f32<T>(v[0]);
    }
  }
};

struct MoveArgs {
  const void* a;       // tokens' rows (gather), or pairs' rows
  const void* b;       // combine_grad: the pairs' rows z
  const int32_t* pos;  // [T][k]
  const float* w;      // [T][k], or nullptr
  void* out;
  float* dw;
  int T, k, H, n_rows;
};

// Copies each token's row to the rows of its pairs.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) gather_kernel(const MoveArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t t = blockIdx.x;
  constexpr int N = Piece<T, VEC>::N;
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * N; c < a.H; c += gridDim.y * blockDim.x * N) {
    Piece<T, VEC> p;
    p.load(static_cast<const T*>(a.a) + t * a.H + c);
    for (int j = 0; j < a.k; ++j) {
      const int r = __ldg(a.pos + t * a.k + j);
      if (static_cast<uint32_t>(r) < static_cast<uint32_t>(a.n_rows)) {
        p.store(static_cast<T*>(a.out) + static_cast<size_t>(r) * a.H + c);
      }
    }
  }
}

// out[t] = sum_j w[t][j] a[pos[t][j]], slots ascending, fp32 (w nullptr: 1).
// Slots without a row add nothing and their weight is not used.
template <typename T, bool VEC, bool WEIGHTED, typename OutT>
__global__ void __launch_bounds__(256) combine_kernel(const MoveArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t t = blockIdx.x;
  constexpr int N = Piece<T, VEC>::N, U = 8;  // slots in flight
  for (int c = (blockIdx.y * blockDim.x + threadIdx.x) * N; c < a.H; c += gridDim.y * blockDim.x * N) {
    float s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 0.f;
    for (int j0 = 0; j0 < a.k; j0 += U) {
      typename Piece<T, VEC>::Raw p[U];
      float w[U];
      bool ok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = j0 + u < a.k ? __ldg(a.pos + t * a.k + j0 + u) : -1;
        ok[u] = static_cast<uint32_t>(r) < static_cast<uint32_t>(a.n_rows);
        if (ok[u]) p[u] = Piece<T, VEC>::raw(static_cast<const T*>(a.a) + static_cast<size_t>(r) * a.H + c);
        if (WEIGHTED && ok[u]) w[u] = __ldg(a.w + t * a.k + j0 + u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!ok[u]) continue;
        Piece<T, VEC> x;
        x.unpack(p[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = WEIGHTED ? fmaf(w[u], x.v[i], s[i]) : s[i] + x.v[i];
      }
    }
    OutT* o = static_cast<OutT*>(a.out) + t * a.H + c;
    if constexpr (VEC) {
      constexpr int PER = 16 / sizeof(OutT);
      if constexpr (N % PER == 0) {
#pragma unroll
        for (int q = 0; q < N / PER; ++q) {
          uint4 u;
          OutT* x = reinterpret_cast<OutT*>(&u);
#pragma unroll
          for (int i = 0; i < PER; ++i) x[i] = from_f32<OutT>(s[q * PER + i]);
          reinterpret_cast<uint4*>(o)[q] = u;
        }
      } else {  // fp32 rows to a 16-bit type: 4 values, 8 bytes
        uint2 u;
        OutT* x = reinterpret_cast<OutT*>(&u);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = from_f32<OutT>(s[i]);
        *reinterpret_cast<uint2*>(o) = u;
      }
    } else {
      o[0] = from_f32<OutT>(s[0]);
    }
  }
}

// A warp per pair: out[pos] = w dy[t] and dw = <dy[t], z[pos]> (four sums per
// lane in fp32, then a shuffle tree).  The k pairs of a token sit in neighbouring
// warps, so dy[t] is read from memory once.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) combine_grad_kernel(const MoveArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const long pair = static_cast<long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (pair >= static_cast<long>(a.T) * a.k) return;
  const int r = __ldg(a.pos + pair);
  float dot = 0.f;
  if (static_cast<uint32_t>(r) < static_cast<uint32_t>(a.n_rows)) {
    constexpr int N = Piece<T, VEC>::N;
    const T* dy = static_cast<const T*>(a.a) + static_cast<size_t>(pair / a.k) * a.H;
    const T* z = static_cast<const T*>(a.b) + static_cast<size_t>(r) * a.H;
    T* dz = static_cast<T*>(a.out) + static_cast<size_t>(r) * a.H;
    const float w = __ldg(a.w + pair);
    constexpr int U = VEC ? 4 : 8;  // pieces of both rows in flight
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = lane * N; c0 < a.H; c0 += 32 * N * U) {
      typename Piece<T, VEC>::Raw rg[U], rx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * N * u;
        if (c < a.H) {
          rg[u] = Piece<T, VEC>::raw(dy + c);
          rx[u] = Piece<T, VEC>::raw(z + c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + 32 * N * u;
        if (c < a.H) {
          Piece<T, VEC> g, x;
          g.unpack(rg[u]);
          x.unpack(rx[u]);
#pragma unroll
          for (int i = 0; i < N; ++i) part[(VEC ? i : u) & 3] = fmaf(g.v[i], x.v[i], part[(VEC ? i : u) & 3]);
#pragma unroll
          for (int i = 0; i < N; ++i) g.v[i] *= w;
          g.store(dz + c);
        }
      }
    }
    dot = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
  }
  if (lane == 0) a.dw[pair] = dot;
}

bool vectors(int H, size_t es, std::initializer_list<const void*> ps) {
  if (H * es % 16 != 0) return false;
  for (const void* p : ps) {
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return false;
  }
  return true;
}

// Threads of a block along a row, and blocks per row.
void row_shape(int pieces, int T, dim3& grid, dim3& block) {
  const int threads = std::min(256, (pieces + 31) / 32 * 32);
  grid = dim3(T, std::min(65535, (pieces + threads - 1) / threads));
  block = dim3(threads);
}

template <typename F>
cudaError_t by_type(hq_dtype d, F&& f) {
  switch (d) {
    case HQ_F16: return f(__half{});
    case HQ_BF16: return f(__nv_bfloat16{});
    default: return f(float{});
  }
}

}  // namespace

static int sort_tile(long pairs) {
  if (pairs <= kOneTile) return kOneTile;
  const long t = (pairs + kMaxTiles - 1) / kMaxTiles;
  return static_cast<int>(std::max<long>(kMinTile, (t + kMinTile - 1) / kMinTile * kMinTile));
}
static int sort_tiles(long pairs) {
  const int t = sort_tile(pairs);
  return static_cast<int>(std::max<long>(1, (pairs + t - 1) / t));
}

// Room for every smaller number of pairs too.
size_t sort_workspace_bytes(long pairs, int E) {
  const long tiles = pairs > kOneTile ? std::min<long>(kMaxTiles, (pairs + kMinTile - 1) / kMinTile) : 0;
  return 256 + (static_cast<size_t>(tiles) * E * 4 + 255) / 256 * 256;
}

int sort_launches(long pairs) { return sort_tiles(pairs) > 1 ? 2 : 1; }

bool sort_supported(long pairs, int E, int align) {
  return E <= kMaxExperts && pairs <= kMaxPairs && pairs + static_cast<long>(E) * (align - 1) < 0x7fffffffl;
}

cudaError_t launch_sort(const int32_t* ids, int pairs, int E, int align, int32_t* pos, int32_t* offsets,
                        int32_t* counts, void* ws, cudaStream_t st) {
  SortArgs a{ids,     pairs,  E, align, sort_tiles(pairs), sort_tile(pairs), 32 - __builtin_clz(E), pos, offsets, counts,
             reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 256)};
  const size_t smem = static_cast<size_t>(sort_warps(E)) * E * 4;
  if (a.tiles > 1) {
    const cudaError_t e = launch_pdl(sort_count_kernel, dim3(a.tiles), dim3(kSortThreads), smem, st, true, a);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(sort_place_kernel, dim3(a.tiles), dim3(kSortThreads), smem, st, true, a);
}

cudaError_t launch_combine(hq_dtype zd, hq_dtype yd, const void* z, const int32_t* pos, const float* w, void* y,
                           int T, int k, int H, int n_rows, cudaStream_t st) {
  MoveArgs a{z, nullptr, pos, w, y, nullptr, T, k, H, n_rows};
  return by_type(zd, [&](auto zt) {
    return by_type(yd, [&](auto yt) -> cudaError_t {
      using Z = decltype(zt);
      using Y = decltype(yt);
      // a sum of 16-bit rows in fp32, or of fp32 rows in any type
      if constexpr (!std::is_same_v<Z, Y> && !std::is_same_v<Z, float> && !std::is_same_v<Y, float>) {
        return cudaErrorInvalidValue;
      } else {
        const bool vec = vectors(H, sizeof(Z), {z, y});
        dim3 grid, block;
        row_shape(vec ? H / static_cast<int>(16 / sizeof(Z)) : H, T, grid, block);
        if (w != nullptr) {
          return vec ? launch_pdl(combine_kernel<Z, true, true, Y>, grid, block, 0, st, true, a)
                     : launch_pdl(combine_kernel<Z, false, true, Y>, grid, block, 0, st, true, a);
        }
        return vec ? launch_pdl(combine_kernel<Z, true, false, Y>, grid, block, 0, st, true, a)
                   : launch_pdl(combine_kernel<Z, false, false, Y>, grid, block, 0, st, true, a);
      }
    });
  });
}

static cudaError_t launch_gather(hq_dtype d, const MoveArgs& a, cudaStream_t st) {
  return by_type(d, [&](auto t) {
    using X = decltype(t);
    const bool vec = vectors(a.H, sizeof(X), {a.a, a.out});
    dim3 grid, block;
    row_shape(vec ? a.H / static_cast<int>(16 / sizeof(X)) : a.H, a.T, grid, block);
    return vec ? launch_pdl(gather_kernel<X, true>, grid, block, 0, st, true, a)
               : launch_pdl(gather_kernel<X, false>, grid, block, 0, st, true, a);
  });
}

static cudaError_t launch_combine_grad(hq_dtype d, const MoveArgs& a, cudaStream_t st) {
  const long pairs = static_cast<long>(a.T) * a.k;
  return by_type(d, [&](auto t) {
    using X = decltype(t);
    const dim3 grid(static_cast<unsigned>((pairs + 7) / 8));
    return vectors(a.H, sizeof(X), {a.a, a.b, a.out})
               ? launch_pdl(combine_grad_kernel<X, true>, grid, dim3(256), 0, st, true, a)
               : launch_pdl(combine_grad_kernel<X, false>, grid, dim3(256), 0, st, true, a);
  });
}

// What every row mover checks: types, sizes, pos, and pointers aligned to
// their element.
static hq_status check_move(hq_dtype d, int T, int k, int H, int n_rows) {
  if (d < HQ_F16 || d > HQ_F32) return HQ_ERR_INVALID_ARG;
  if (T < 0 || k < 1 || H < 1 || n_rows < 0) return HQ_ERR_INVALID_ARG;
  if (k > 32 || static_cast<long>(T) * k > 0x7fffffffl || H > (1 << 24)) return HQ_ERR_UNSUPPORTED;
  return HQ_OK;
}
static bool bad(const void* p, uintptr_t a) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0;
}

}  // namespace route
}  // namespace hq

using namespace hq;

extern "C" {

size_t hq_moe_sort_workspace_size(int T, int k, int n_experts) {
  if (T < 0 || k < 1 || k > 32 || n_experts < 1 || !route::sort_supported(static_cast<long>(T) * k, n_experts, 1)) {
    return 0;
  }
  return route::sort_workspace_bytes(static_cast<long>(T) * k, n_experts);
}

hq_status hq_moe_sort(const int32_t* topk_ids, int T, int k, int n_experts, int align, int32_t* pos,
                      int32_t* offsets, int32_t* counts, void* workspace, size_t ws_bytes, hq_stream_t stream) {
  if (T < 0 || k < 1 || n_experts < 1 || align < 1) return HQ_ERR_INVALID_ARG;
  const long pairs = static_cast<long>(T) * k;
  if (k > 32 || align > 4096 || !route::sort_supported(pairs, n_experts, align)) return HQ_ERR_UNSUPPORTED;
  if ((pairs > 0 && (route::bad(topk_ids, 4) || route::bad(pos, 4))) || route::bad(offsets, 4) ||
      route::bad(counts, 4)) {
    return HQ_ERR_INVALID_ARG;
  }
  if (route::bad(workspace, 256) || ws_bytes < route::sort_workspace_bytes(pairs, n_experts)) {
    return HQ_ERR_WORKSPACE;
  }
  return from_cuda(route::launch_sort(topk_ids, static_cast<int>(pairs), n_experts, align, pos, offsets, counts,
                                      workspace, reinterpret_cast<cudaStream_t>(stream)));
}

hq_status hq_moe_gather(const void* x, hq_dtype dtype, const int32_t* pos, int T, int k, int H, void* rows,
                        int n_rows, hq_stream_t stream) {
  const hq_status ok = route::check_move(dtype, T, k, H, n_rows);
  if (ok != HQ_OK) return ok;
  if (T == 0 || n_rows == 0) return HQ_OK;
  const uintptr_t es = dtype == HQ_F32 ? 4 : 2;
  if (route::bad(x, es) || route::bad(pos, 4) || route::bad(rows, es)) return HQ_ERR_INVALID_ARG;
  return from_cuda(route::launch_gather(dtype, {x, nullptr, pos, nullptr, rows, nullptr, T, k, H, n_rows},
                                        reinterpret_cast<cudaStream_t>(stream)));
}

hq_status hq_moe_combine(const void* rows, hq_dtype dtype, int n_rows, const int32_t* pos, const float* topk_w,
                         int T, int k, int H, void* y, hq_dtype y_dtype, hq_stream_t stream) {
  const hq_status ok = route::check_move(dtype, T, k, H, n_rows);
  if (ok != HQ_OK) return ok;
  if (y_dtype < HQ_F16 || y_dtype > HQ_F32) return HQ_ERR_INVALID_ARG;
  if (y_dtype != dtype && dtype != HQ_F32 && y_dtype != HQ_F32) return HQ_ERR_UNSUPPORTED;
  if (T == 0) return HQ_OK;
  const uintptr_t es = dtype == HQ_F32 ? 4 : 2, ys = y_dtype == HQ_F32 ? 4 : 2;
  if ((n_rows > 0 && route::bad(rows, es)) || route::bad(pos, 4) || route::bad(y, ys) ||
      (reinterpret_cast<uintptr_t>(topk_w) & 3) != 0) {
    return HQ_ERR_INVALID_ARG;
  }
  return from_cuda(route::launch_combine(dtype, y_dtype, rows, pos, topk_w, y, T, k, H, n_rows,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

hq_status hq_moe_combine_grad(const void* dy, hq_dtype dtype, const void* rows, int n_rows, const int32_t* pos,
                              const float* topk_w, int T, int k, int H, void* drows, float* dw,
                              hq_stream_t stream) {
  const hq_status ok = route::check_move(dtype, T, k, H, n_rows);
  if (ok != HQ_OK) return ok;
  if (T == 0) return HQ_OK;
  const uintptr_t es = dtype == HQ_F32 ? 4 : 2;
  if (route::bad(dy, es) || (n_rows > 0 && (route::bad(rows, es) || route::bad(drows, es))) ||
      route::bad(pos, 4) || route::bad(topk_w, 4) || route::bad(dw, 4)) {
    return HQ_ERR_INVALID_ARG;
  }
  return from_cuda(route::launch_combine_grad(dtype, {dy, rows, pos, topk_w, drows, dw, T, k, H, n_rows},
                                              reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
