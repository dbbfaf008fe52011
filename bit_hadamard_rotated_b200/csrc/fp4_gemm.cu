// fp4_gemm.cu -- products of microscaled 4-bit matrices on the 5th-generation
// tensor cores: hq_fp4_matmul, hq_fp4_linear and the two products of
// hq_fp4_experts.
//
//   y[n][m] = ts_w ts_a sum_k (c_w s_w)[m][k] (c_a s_a)[n][k]
//
// tcgen05.mma takes E2M1 operands from shared memory and their block scales
// from tensor memory and multiplies them in: no value is decoded anywhere.
// Weights are the M side (128 rows a tile), tokens the N side (16 to 256), so
// a token block of any size streams the weights once and the epilogue's lanes
// run along an output row.
//
// One CTA walks a list of (tile, K range) items.  Per 256 values of K it needs
// 16 KB of weight codes (one TMA box, 128-byte swizzle), the tokens' codes,
// and the scale tiles (bulk copies: they lie in memory as tcgen05.cp wants
// them), all on one mbarrier per ring slot.
//   warp 0   producer: one thread issues the copies
//   warp 1   one thread moves the slot's scales to tensor memory and issues
//            the MMAs (K = 64 each); their commit frees the slot
//   others   epilogue: tensor memory to registers, alpha, one rounding, y
// Two accumulators where they fit (up to 128 tokens), so the next tile's MMAs
// run under the epilogue.
//
// Few tiles: the (tile, chunk) units are split evenly over the CTAs, so a tile
// may be shared by several; each leaves its partial sums in the workspace and
// the last to arrive adds them in CTA order (the result does not depend on
// who is last).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fp4.cuh"
#include "hq_common.cuh"
#include "hq_internal.h"
#include "hq_io.cuh"
#include "hq_launch.cuh"
#include "route.cuh"
#include "tcgen05.cuh"

namespace hq {
namespace fp4 {
namespace {

constexpr int kM = 128;      // weight rows per tile
constexpr int kChunk = 256;  // values of K per ring slot (128 bytes a row)
constexpr int kWBytes = kM * kChunk / 2;

// ------------------------------------------------------------------ PTX

// Scale tile (512 bytes) to four tensor-memory columns, in all four lane
// quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = tc::smem_desc(smem, 0, 128);
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D (+)= (A sA) (B sB), K = 64, E2M1, A and B K-major in shared memory.
template <int FMT>
__device__ __forceinline__ void tc_mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                              uint32_t sb, uint32_t accumulate) {
  if constexpr (FMT == HQ_FP4_NV) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  }
}

// Instruction descriptor of the block-scaled kinds: E2M1 operands (1 at bits
// 7 and 10), N / 8 at 17, the scales' type at 23 (0 E4M3, 1 E8M0), M / 16 at
// 24; the scales' byte within its word at 29 (A) and 4 (B).
__device__ __forceinline__ constexpr uint32_t idesc_fp4(int fmt, int n, int sf_id) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (fmt == HQ_FP4_MX ? 1u << 23 : 0u) | (static_cast<uint32_t>(kM >> 4) << 24) |
         (static_cast<uint32_t>(sf_id) << 29) | (static_cast<uint32_t>(sf_id) << 4);
}

// Shared-memory descriptor of a K-major operand in the 128-byte swizzle: rows
// of 128 bytes, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// ------------------------------------------------------------------ plan

template <int FMT, int NT>
struct Shape {
  static constexpr int kTiles = kChunk / (FMT == HQ_FP4_NV ? 64 : 128);  // scale tiles per chunk
  static constexpr int kSfA = kTiles * 512;
  static constexpr int kRowTiles = NT > 128 ? NT / 128 : 1;              // token scale tiles
  static constexpr int kSfB = kRowTiles * kTiles * 512;
  static constexpr int kABytes = NT * kChunk / 2;
  static constexpr int kSlot = kWBytes + kABytes + kSfA + kSfB;
  static constexpr int kAccs = NT <= 128 ? 2 : 1;
  static constexpr int kSfCols = kTiles * 4 * (1 + kRowTiles);           // one slot's scales
  static constexpr int kSfSets = 2;
  static constexpr int kColsNeeded = kAccs * NT + kSfSets * kSfCols;
  static constexpr int kCols = kColsNeeded <= 128 ? 128 : kColsNeeded <= 256 ? 256 : 512;
  static constexpr int kEpiWarps = NT > 128 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStages = NT <= 64 ? 4 : NT <= 128 ? 5 : 4;
  static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kSlot + 512;
  static_assert(kColsNeeded <= 512, "tensor memory");
  static_assert(kSlot % 1024 == 0, "swizzle atoms");
};

struct GemmArgs {
  const uint8_t* wsf;  // weight scale tiles
  const uint8_t* asf;  // token scale tiles
  const float* wts;
  const float* ats;
  int wkb;             // scale tiles along K
  int a_row_tiles;     // token scale row tiles
  int M, N, C;         // weight rows (of one expert), tokens, chunks of K
  int k_steps;         // MMAs of 64 over the whole of K
  int mt, nt;          // tiles
  int units;           // split: mt * nt * C (whole tiles: 0)
  void* y;
  int y_dtype;
  size_t ldy;
  uint32_t* status;
  uint32_t* counters;  // split: per CTA, zero between calls
  float* part;         // split: 2 slots of [NT][128] per CTA
  // grouped: the experts' row segments; tiles are (expert, token tile, m tile)
  const int32_t* offsets;
  const int32_t* counts;
  int E, n_wts;
  int early;           // the weights may be read before the preceding kernel ends
};

// One item of a CTA's list: a tile and its chunks [c0, c1).
struct Item {
  int m0, n0, n_valid;  // first weight row in its expert, first token row, token rows
  int w_row;            // first weight row in the matrix
  int e;
  int c0, c1;
};

template <int NT, bool GROUPED>
struct Walk {
  int u, end, step, tile0;
  // grouped
  int e, left, first;  // current expert, its first tile's index
  __device__ __forceinline__ void start(const GemmArgs& a) {
    if constexpr (GROUPED) {
      u = blockIdx.x;
      step = gridDim.x;
      e = 0;
      first = 0;
    } else if (a.units > 0) {
      u = static_cast<int>(static_cast<long>(a.units) * blockIdx.x / gridDim.x);
      end = static_cast<int>(static_cast<long>(a.units) * (blockIdx.x + 1) / gridDim.x);
    } else {
      u = blockIdx.x;
      end = a.mt * a.nt;
      step = gridDim.x;
    }
  }
  // The next item; false at the end.  n tiles fastest: CTAs that run together
  // share weight tiles in L2.
  __device__ __forceinline__ bool next(const GemmArgs& a, Item& it) {
    if constexpr (GROUPED) {
      while (e < a.E) {
        const int cnt = __ldg(a.counts + e);
        const int tiles = (cnt + NT - 1) / NT * a.mt;
        if (u < first + tiles) {
          const int t = u - first, nti = t / a.mt, mi = t - nti * a.mt;
          it.m0 = mi * kM;
          it.n0 = __ldg(a.offsets + e) + nti * NT;
          it.n_valid = min(NT, cnt - nti * NT);
          it.w_row = e * a.M + it.m0;
          it.e = e;
          it.c0 = 0;
          it.c1 = a.C;
          u += step;
          return true;
        }
        first += tiles;
        ++e;
      }
      return false;
    } else {
      if (u >= end) return false;
      int tile = u;
      it.c0 = 0;
      it.c1 = a.C;
      if (a.units > 0) {
        tile = u / a.C;
        it.c0 = u - tile * a.C;
        it.c1 = min(a.C, it.c0 + end - u);
        u += it.c1 - it.c0;
      } else {
        u += step;
      }
      const int mi = tile / a.nt, ni = tile - mi * a.nt;
      it.m0 = mi * kM;
      it.n0 = ni * NT;
      it.n_valid = min(NT, a.N - it.n0);
      it.w_row = it.m0;
      it.e = 0;
      return true;
    }
  }
};

template <typename T>
__device__ __forceinline__ void put(void* y, size_t i, float v) {
  static_cast<T*>(y)[i] = from_f32<T>(v);
}

// ------------------------------------------------------------------ kernel

template <int FMT, int NT, bool GROUPED>
__global__ void __launch_bounds__(Shape<FMT, NT>::kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                const GemmArgs a) {
  using S = Shape<FMT, NT>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ST * S::kSlot);
  uint64_t* empty = full + ST;
  uint64_t* dfull = empty + ST;
  uint64_t* dempty = dfull + S::kAccs;
  uint64_t* epi = dempty + S::kAccs;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(epi + 1);
  uint32_t* flag = tslot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < S::kAccs; ++i) {
      mbar_init(dfull + i, 1);
      mbar_init(dempty + i, S::kEpiWarps);
    }
    mbar_init(epi, S::kEpiWarps);
    fence_mbar_init();
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&amap);
  }
  if (warp == 1) {
    tc::tmem_alloc(tslot, S::kCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t sf_cols = tmem + S::kAccs * NT;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      const bool early = !GROUPED && a.early != 0;
      if (!early) pdl_wait();
      Walk<NT, GROUPED> w;
      w.start(a);
      Item it;
      int slot = 0, turn = 0;
      // With early weights: the first ring of weight copies goes out before the
      // wait, the token copies of the same slots after it.
      Walk<NT, GROUPED> w2 = w;
      Item it2;
      int ahead = 0;
      auto bytes_of = [&](const Item& t, int c, int& tiles, int& row_tiles, int& a_rows) {
        tiles = min(S::kTiles, a.wkb - c * S::kTiles);
        row_tiles = min(S::kRowTiles, a.a_row_tiles - (t.n0 >> 7));
        a_rows = GROUPED ? (t.n_valid + 15) / 16 * 16 : NT;
        return static_cast<uint32_t>(kWBytes + a_rows * 128 + tiles * 512 * (1 + row_tiles));
      };
      auto weights = [&](const Item& t, int c, int s) {
        int tiles, row_tiles, a_rows;
        const uint32_t bytes = bytes_of(t, c, tiles, row_tiles, a_rows);
        uint8_t* p = ring + s * S::kSlot;
        mbar_arrive_expect_tx(full + s, bytes);
        tma_load_2d(p, &wmap, c * (kChunk / 2), t.w_row, full + s);
        bulk_g2s(p + kWBytes + S::kABytes, a.wsf + (static_cast<size_t>(t.w_row >> 7) * a.wkb + c * S::kTiles) * 512,
                 tiles * 512, full + s);
      };
      auto tokens = [&](const Item& t, int c, int s) {
        int tiles, row_tiles, a_rows;
        bytes_of(t, c, tiles, row_tiles, a_rows);
        uint8_t* p = ring + s * S::kSlot;
        if constexpr (GROUPED) {
          for (int r = 0; r < a_rows; r += 16) {
            tma_load_2d(p + kWBytes + r * 128, &amap, c * (kChunk / 2), t.n0 + r, full + s);
          }
        } else {
          tma_load_2d(p + kWBytes, &amap, c * (kChunk / 2), t.n0, full + s);
        }
        for (int r = 0; r < row_tiles; ++r) {
          bulk_g2s(p + kWBytes + S::kABytes + S::kSfA + r * S::kSfA,
                   a.asf + (static_cast<size_t>((t.n0 >> 7) + r) * a.wkb + c * S::kTiles) * 512, tiles * 512,
                   full + s);
        }
      };
      if (early) {
        bool more = true;
        while (more && ahead < ST) {
          more = w2.next(a, it2);
          if (!more) break;
          for (int c = it2.c0; c < it2.c1 && ahead < ST; ++c) weights(it2, c, ahead++);
        }
        pdl_wait();
      }
      int n = 0;  // chunks so far
      while (ok && w.next(a, it)) {
        for (int c = it.c0; c < it.c1; ++c) {
          if (n >= ST && !mbar_wait(empty + slot, turn ^ 1)) {
            ok = false;
            break;
          }
          if (n >= ahead) weights(it, c, slot);
          tokens(it, c, slot);
          ++n;
          if (++slot == ST) {
            slot = 0;
            turn ^= 1;
          }
        }
      }
      pdl_launch_dependents();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      if constexpr (GROUPED) pdl_wait();  // it reads the segments
      Walk<NT, GROUPED> w;
      w.start(a);
      Item it;
      int slot = 0, par = 0, set = 0, acc = 0, accn = 0;
      while (ok && w.next(a, it)) {
        const uint32_t d = tmem + acc * NT;
        if (accn >= S::kAccs && !mbar_wait(dempty + acc, (accn / S::kAccs - 1) & 1)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const int n_mma = (it.n_valid + 15) / 16 * 16;
        for (int c = it.c0; c < it.c1; ++c) {
          if (!mbar_wait(full + slot, par)) {
            ok = false;
            break;
          }
          tc::tc_fence_after();
          const uint32_t p = smem_u32(ring + slot * S::kSlot);
          const uint32_t sfa = sf_cols + set * S::kSfCols, sfb = sfa + S::kTiles * 4;
          const uint32_t sp = p + kWBytes + S::kABytes;
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t) {
            tc_copy_scales(sfa + 4 * t, sp + 512 * t);
#pragma unroll
            for (int r = 0; r < S::kRowTiles; ++r) {
              tc_copy_scales(sfb + 4 * (t * S::kRowTiles + r), sp + S::kSfA * (1 + r) + 512 * t);
            }
          }
          const uint64_t da = desc_sw128(p), db = desc_sw128(p + kWBytes);
          // the tokens' rows within their scale tile: 0 or 64 (two columns)
          const uint32_t half = NT < 128 ? ((it.n0 & 127) >> 5) : 0;
          const int steps = min(4, a.k_steps - 4 * c);
          for (int s = 0; s < steps; ++s) {
            const int t = FMT == HQ_FP4_NV ? s : s >> 1, id = FMT == HQ_FP4_NV ? 0 : 2 * (s & 1);
            tc_mma_scaled<FMT>(d, da + 2 * s, db + 2 * s, idesc_fp4(FMT, n_mma, id), sfa + 4 * t,
                               sfb + 4 * t * S::kRowTiles + half, (c > it.c0 || s > 0) ? 1u : 0u);
          }
          tc::tc_commit(empty + slot);
          set ^= 1;
          if (++slot == ST) {
            slot = 0;
            par ^= 1;
          }
        }
        if (!ok) break;
        tc::tc_commit(dfull + acc);
        ++accn;
        acc = accn % S::kAccs;
      }
    }
  } else {
    pdl_wait();
    const int ew = warp - 2, quarter = warp & 3;
    constexpr int kParts = S::kEpiWarps / 4;  // warps that share a lane quarter split the columns
    const int col0 = (ew >> 2) * (NT / kParts), col1 = col0 + NT / kParts;
    const int mrow = quarter * 32 + lane;
    const float ats = a.ats != nullptr ? __ldg(a.ats) : 1.f;
    Walk<NT, GROUPED> w;
    w.start(a);
    Item it;
    int acc = 0, accn = 0, epar = 0;
    auto meet = [&]() {  // all epilogue warps, bounded
      __syncwarp();
      if (lane == 0) mbar_arrive(epi);
      const bool r = __all_sync(~0u, mbar_wait(epi, epar));
      epar ^= 1;
      return r;
    };
    while (ok && w.next(a, it)) {
      if (!__all_sync(~0u, mbar_wait(dfull + acc, (accn / S::kAccs) & 1))) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const uint32_t d = tmem + acc * NT + (static_cast<uint32_t>(quarter * 32) << 16);
      const float alpha = (a.wts != nullptr ? __ldg(a.wts + (a.n_wts > 1 ? it.e : 0)) : 1.f) * ats;
      const bool whole = it.c0 == 0 && it.c1 == a.C;
      const int m = it.m0 + mrow;
      if (whole) {
        for (int c = col0; c < col1 && c < it.n_valid; c += 16) {
          uint32_t v[16];
          tc::tc_ld16(d + c, v);
          tc::tc_wait_ld();
          tc::tc_tie16(v);
          if (m < a.M) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c + i < it.n_valid) {
                const size_t o = static_cast<size_t>(it.n0 + c + i) * a.ldy + m;
                const float f = __uint_as_float(v[i]) * alpha;
                if (a.y_dtype == HQ_BF16) put<__nv_bfloat16>(a.y, o, f);
                else if (a.y_dtype == HQ_F16) put<__half>(a.y, o, f);
                else put<float>(a.y, o, f);
              }
            }
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dempty + acc);
      } else if constexpr (!GROUPED) {
        // a tile shared by CTAs i0 .. i1: the units [t C, t C + C)
        const int t = (it.m0 / kM) * a.nt + it.n0 / NT;
        const long first = static_cast<long>(t) * a.C, last = first + a.C - 1;
        const int i0 = static_cast<int>(((first + 1) * gridDim.x - 1) / a.units);
        const int i1 = static_cast<int>(((last + 1) * gridDim.x - 1) / a.units);
        const size_t part_size = static_cast<size_t>(NT) * kM;
        // a CTA's second slot is for the tile that it begins
        float* mine = a.part + (2 * static_cast<size_t>(blockIdx.x) + (it.c0 == 0 ? 1 : 0)) * part_size;
        for (int c = col0; c < col1 && c < it.n_valid; c += 16) {
          uint32_t v[16];
          tc::tc_ld16(d + c, v);
          tc::tc_wait_ld();
          tc::tc_tie16(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) __stcg(mine + (c + i) * kM + mrow, __uint_as_float(v[i]));
        }
        tc::tc_fence_before();
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(dempty + acc);
        if (!meet()) {
          ok = false;
          break;
        }
        if (ew == 0 && lane == 0) {
          __threadfence();
          *flag = atomicAdd(a.counters + i0, 1u) == static_cast<uint32_t>(i1 - i0) ? 1u : 0u;
        }
        if (!meet()) {
          ok = false;
          break;
        }
        if (*reinterpret_cast<volatile uint32_t*>(flag) != 0) {
          __threadfence();
          for (int c = col0; c < col1 && c < it.n_valid; ++c) {
            float s = 0.f;
            for (int i = i0; i <= i1; ++i) {
              s += __ldcg(a.part + (2 * static_cast<size_t>(i) + (i == i0 ? 1 : 0)) * part_size + c * kM + mrow);
            }
            if (m < a.M) {
              const size_t o = static_cast<size_t>(it.n0 + c) * a.ldy + m;
              const float f = s * alpha;
              if (a.y_dtype == HQ_BF16) put<__nv_bfloat16>(a.y, o, f);
              else if (a.y_dtype == HQ_F16) put<__half>(a.y, o, f);
              else put<float>(a.y, o, f);
            }
          }
          if (ew == 0 && lane == 0) a.counters[i0] = 0;
        }
        // the flag is read before it is written again: the next tile's first
        // meeting comes between
      }
      ++accn;
      acc = accn % S::kAccs;
    }
  }
  if (!ok) record_error(a.status, HQ_DEV_TIMEOUT);
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, S::kCols);
}

// ------------------------------------------------------------------ host

constexpr size_t kStatusBytes = 256;
constexpr size_t kCounterBytes = 1024;  // one word per CTA of a split grid
constexpr int kMaxGrid = static_cast<int>(kCounterBytes / 4);

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// How a dense product runs: tokens per tile, CTAs, and the (tile, chunk)
// units if they are split evenly (0: whole tiles).
struct Plan {
  int nt_size, mt, nt, C, grid, units;
};

int tokens_per_tile(int N) { return N <= 32 ? 32 : N <= 64 ? 64 : N <= 128 ? 128 : 256; }

// Room for every plan of up to N tokens: a workspace for N serves all smaller
// batches too.
size_t part_bound(int N, int K) {
  return K <= kChunk ? 0
                     : static_cast<size_t>(std::min(sm_count(), kMaxGrid)) * 2 * tokens_per_tile(N) * kM * sizeof(float);
}

Plan plan_of(int M, int N, int K) {
  Plan p{};
  p.C = (K + kChunk - 1) / kChunk;
  p.mt = (M + kM - 1) / kM;
  p.nt_size = tokens_per_tile(N);
  p.nt = (N + p.nt_size - 1) / p.nt_size;
  const int sms = std::min(sm_count(), kMaxGrid);
  const long tiles = static_cast<long>(p.mt) * p.nt;
  const long units = tiles * p.C;
  if (tiles % sms != 0 && tiles < 4l * sms && p.C > 1) {
    p.grid = static_cast<int>(std::min<long>(sms, std::max(tiles, units / 2)));
    p.units = static_cast<int>(units);
  } else {
    p.grid = static_cast<int>(std::min<long>(sms, tiles));
  }
  return p;
}

template <int FMT, int NT, bool GROUPED>
cudaError_t gemm_launch(const CUtensorMap& wmap, const CUtensorMap& amap, const GemmArgs& a, int grid,
                        cudaStream_t st) {
  using S = Shape<FMT, NT>;
  return launch_pdl(gemm_kernel<FMT, NT, GROUPED>, dim3(grid), dim3(S::kThreads), S::kSmem, st, true, wmap, amap, a);
}

template <int FMT>
cudaError_t dense_launch(int nt, const CUtensorMap& wmap, const CUtensorMap& amap, const GemmArgs& a, int grid,
                         cudaStream_t st) {
  switch (nt) {
    case 32: return gemm_launch<FMT, 32, false>(wmap, amap, a, grid, st);
    case 64: return gemm_launch<FMT, 64, false>(wmap, amap, a, grid, st);
    case 128: return gemm_launch<FMT, 128, false>(wmap, amap, a, grid, st);
    default: return gemm_launch<FMT, 256, false>(wmap, amap, a, grid, st);
  }
}

cudaError_t code_map(CUtensorMap* map, const uint8_t* codes, long rows, int K, int box_rows) {
  return tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K / 2),
                       static_cast<uint64_t>(rows), static_cast<uint64_t>(K / 2), kChunk / 2, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// y = W a for a packed token matrix; part and counters as the plan needs them.
cudaError_t launch_matmul(const hq_fp4_matrix* w, const uint8_t* codes, const uint8_t* scales, const float* ats,
                          int N, void* y, hq_dtype yd, size_t ldy, uint8_t* ws, uint8_t* part, bool early,
                          cudaStream_t st) {
  const Plan p = plan_of(w->rows, N, w->K);
  CUtensorMap wmap, amap;
  cudaError_t e = code_map(&wmap, w->codes, w->rows, w->K, kM);
  if (e != cudaSuccess) return e;
  e = code_map(&amap, codes, N, w->K, p.nt_size);
  if (e != cudaSuccess) return e;
  GemmArgs a{};
  a.wsf = w->scales;
  a.asf = scales;
  a.wts = w->tensor_scale;
  a.n_wts = 1;
  a.ats = ats;
  a.wkb = scale_tiles(w->format, w->K);
  a.a_row_tiles = (N + 127) / 128;
  a.M = w->rows;
  a.N = N;
  a.C = p.C;
  a.k_steps = (w->K + 63) / 64;
  a.mt = p.mt;
  a.nt = p.nt;
  a.units = p.units;
  a.y = y;
  a.y_dtype = yd;
  a.ldy = ldy;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kStatusBytes);
  a.part = reinterpret_cast<float*>(part);
  a.early = early ? 1 : 0;
  return w->format == HQ_FP4_NV ? dense_launch<HQ_FP4_NV>(p.nt_size, wmap, amap, a, p.grid, st)
                                : dense_launch<HQ_FP4_MX>(p.nt_size, wmap, amap, a, p.grid, st);
}

// Checks of a product's weights, sizes and output.
hq_status check_product(const hq_fp4_matrix* w, int N, const void* y, hq_dtype yd, size_t ldy) {
  const hq_status ok = check_matrix(w);
  if (ok != HQ_OK) return ok;
  if (w->rows < 1 || N < 0 || yd < HQ_F16 || yd > HQ_F32) return HQ_ERR_INVALID_ARG;
  if (w->tensor_scale != nullptr && w->n_tensor_scales != 1) return HQ_ERR_UNSUPPORTED;
  if (N > (1 << 22)) return HQ_ERR_UNSUPPORTED;
  if (N == 0) return HQ_OK;
  const uintptr_t es = yd == HQ_F32 ? 4 : 2;
  if (y == nullptr || (reinterpret_cast<uintptr_t>(y) & (es - 1)) != 0) return HQ_ERR_INVALID_ARG;
  if (ldy < static_cast<size_t>(w->rows) || ldy > (size_t{1} << 40)) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

bool bad_workspace(const void* ws, size_t bytes, size_t need) {
  return ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255) != 0 || bytes < need;
}

size_t packed_bytes(int fmt, long rows, int K) {
  return align256(static_cast<size_t>(rows) * (K / 2)) + align256(scale_bytes(fmt, rows, K));
}

}  // namespace
}  // namespace fp4
}  // namespace hq

using namespace hq;

extern "C" {

size_t hq_fp4_matmul_workspace_size(const hq_fp4_matrix* w, int n_rows) {
  if (fp4::check_matrix(w) != HQ_OK || w->rows < 1 || n_rows < 0 || n_rows > (1 << 22)) return 0;
  return fp4::kStatusBytes + fp4::kCounterBytes + fp4::part_bound(n_rows, w->K);
}

hq_status hq_fp4_matmul(const hq_fp4_matrix* w, const hq_fp4_matrix* a, void* y, hq_dtype y_dtype, size_t ldy,
                        void* workspace, size_t ws_bytes, hq_stream_t stream) {
  hq_status ok = a == nullptr ? HQ_ERR_INVALID_ARG : fp4::check_product(w, a->rows, y, y_dtype, ldy);
  if (ok != HQ_OK) return ok;
  if (a->rows == 0) return HQ_OK;
  ok = fp4::check_matrix(a);
  if (ok != HQ_OK) return ok;
  if (a->format != w->format || a->K != w->K) return HQ_ERR_INVALID_ARG;
  if (a->tensor_scale != nullptr && a->n_tensor_scales != 1) return HQ_ERR_UNSUPPORTED;
  if (fp4::bad_workspace(workspace, ws_bytes, hq_fp4_matmul_workspace_size(w, a->rows))) return HQ_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return from_cuda(fp4::launch_matmul(w, a->codes, a->scales, a->tensor_scale, a->rows, y, y_dtype, ldy, ws,
                                      ws + fp4::kStatusBytes + fp4::kCounterBytes, false,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t hq_fp4_linear_workspace_size(const hq_fp4_matrix* w, int batch) {
  const size_t b = hq_fp4_matmul_workspace_size(w, batch);
  return b == 0 ? 0 : b + fp4::packed_bytes(w->format, batch, w->K);
}

hq_status hq_fp4_linear(const hq_fp4_matrix* w, const void* x, hq_dtype x_dtype, size_t ldx, int batch,
                        const float* x_scale, void* y, hq_dtype y_dtype, size_t ldy, void* workspace,
                        size_t ws_bytes, hq_stream_t stream) {
  hq_status ok = fp4::check_product(w, batch, y, y_dtype, ldy);
  if (ok != HQ_OK) return ok;
  if (x_scale != nullptr && (w->format != HQ_FP4_NV || (reinterpret_cast<uintptr_t>(x_scale) & 3) != 0)) {
    return HQ_ERR_INVALID_ARG;
  }
  if (batch == 0) return HQ_OK;
  ok = fp4::check_rows(x, x_dtype, ldx, w->K);
  if (ok != HQ_OK) return ok;
  if (fp4::bad_workspace(workspace, ws_bytes, hq_fp4_linear_workspace_size(w, batch))) return HQ_ERR_WORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* codes = ws + fp4::kStatusBytes + fp4::kCounterBytes;
  uint8_t* scales = codes + fp4::align256(static_cast<size_t>(batch) * (w->K / 2));
  uint8_t* part = scales + fp4::align256(fp4::scale_bytes(w->format, batch, w->K));
  const cudaError_t e = fp4::launch_quantize(w->format, x_dtype, x, ldx, batch, w->K, x_scale, codes, scales,
                                             nullptr, nullptr, 1, batch, st);
  if (e != cudaSuccess) return from_cuda(e);
  // The quantiser lets this kernel start only after its own wait, so all that
  // came before it on the stream, the weights' writers too, is complete: the
  // weights may be read at once.
  return from_cuda(fp4::launch_matmul(w, codes, scales, x_scale, batch, y, y_dtype, ldy, ws, part, true, st));
}

int hq_fp4_linear_launches(void) { return 2; }

}  // extern "C"
