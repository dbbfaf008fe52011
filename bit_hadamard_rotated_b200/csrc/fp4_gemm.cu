// fp4_gemm.cu -- products of microscaled 4-bit matrices on the 5th-generation
// tensor cores: hq_fp4_matmul, hq_fp4_linear and the two products of
// hq_fp4_experts.
//
//   y[n][m] = ts_w ts_a sum_k (c_w s_w)[m][k] (c_a s_a)[n][k]
//
// tcgen05.mma takes E2M1 operands from shared memory and their block scales
// from tensor memory and multiplies them in: no value is decoded anywhere.
// Weights are the M side (128 rows a tile), tokens the N side (32 to 128 of
// one CTA, 256 of a pair), so a token block of any size streams the weights once
// and the epilogue's lanes run along an output row.
//
// One CTA walks a list of (tile, K range) items.  Per 256 values of K it needs
// 16 KB of weight codes (one TMA box, 128-byte swizzle), the tokens' codes,
// and the scale tiles (bulk copies), all on one mbarrier per ring slot.
//   warp 0   issues the weights' copies
//   warp 1   moves the slot's scales to tensor memory (tcgen05.cp) and issues
//            the MMAs (K = 64 each) behind them, in order; their commit frees
//            the slot
//   warp 2   issues the tokens' copies
//   others   epilogue: tensor memory to registers, alpha, one rounding, y
// The copies of the scales cost nothing beside the MMAs: 12 of them and 4 MMAs
// of 256 tokens took 512 cycles, the MMAs' own time (through registers, by
// four more warps, they took shared-memory bandwidth from the operands).
// Two accumulators where they fit (up to 128 tokens), so the next tile's MMAs
// run under the epilogue.
//
// Few tiles of a long K: several CTAs take a part of a tile's K each and leave
// their sums in the workspace; the last to arrive adds them in the order of the
// parts (the result does not depend on who is last).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fp4.cuh"
#include "fp4_quant.cuh"
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
constexpr int kTurnRow = 36;  // floats per token of an epilogue transpose (32 and padding)
constexpr int kMaxGroups = 1024;
constexpr int kMaxEpiWarps = 8;   // of a kernel that splits tiles
constexpr int kFusedTokens = 8;   // most tokens of a fused launch (one swizzle atom)
constexpr int kSmemMax = 218 * 1024;  // dynamic; the experts' segments (12 KB) beside it
// More than half an SM's shared memory: no two kernels that hold tensor memory
// share an SM, or one that waits for the other's end could hold what it needs.
constexpr int kSmemMin = 116 * 1024;

// ------------------------------------------------------------------ PTX

// One lane of a converged warp (the same one every time).  The warps that issue
// copies and MMAs run their loops with all lanes on warp-uniform values and
// elect a lane around the instructions only: their operands are then computed
// in uniform registers, which these instructions take.  From one lane in a
// divergent branch every operand is moved over first, and an MMA took about 115
// cycles to issue, a chunk of four with its waits about 900.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A value that all lanes hold alike, by a reduction: its result is in a uniform
// register, so the compiler knows that loops over it do not diverge.  Through a
// shuffle it does not, and an expert tile's walk, waits and operands took 900
// cycles a chunk instead of 650 (when it was changed, 4096 tokens 205 -> 199.5
// us, 32 tokens 59.3 -> 56.4).
__device__ __forceinline__ int uniform(int v) {
  return static_cast<int>(__reduce_or_sync(~0u, static_cast<unsigned>(v)));
}
// A wait that all lanes of a warp agree on.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(~0u, mbar_wait(bar, parity));
}

// The end of a warp that has filled a ring's slots in turn, n times in all:
// waits (within the waits' limit) until its last copies have landed, which they
// have on the usual path, since the MMAs waited for them; but no copy may be in
// flight when a CTA that gave up a wait returns its shared memory.
__device__ __forceinline__ bool drain_slots(uint64_t* full, int stages, int n) {
  for (int i = max(0, n - stages); i < n; ++i) {
    if (!warp_wait(full + i % stages, (i / stages) & 1)) return false;
  }
  return true;
}

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

// What a launch computes: y of one matrix; y of every expert's rows; the
// quantised h = silu(gate) up of every expert's rows; or y of one matrix for a
// few real-valued tokens, quantised on the way.
enum Mode { kDense = 0, kGrouped = 1, kGated = 2, kFused = 3 };

template <int FMT, int NT, int MODE>
struct Shape {
  static constexpr int kW = MODE == kGated ? 2 : 1;                      // weight tiles per slot
  static constexpr int kTiles = kChunk / (FMT == HQ_FP4_NV ? 64 : 128);  // scale tiles per chunk
  static constexpr int kSf = kTiles * 512;                               // one row tile's scales
  static constexpr int kABytes = MODE == kFused ? 0 : NT * kChunk / 2;
  static constexpr int kSfOff = kW * kWBytes + kABytes;                  // scales: weights', then tokens'
  static constexpr int kSlot = kSfOff + (MODE == kFused ? kW : kW + 1) * kSf;
  static constexpr int kAccs = kW * NT <= 128 ? 2 : 1;                   // accumulator sets
  static constexpr int kSfCols = kTiles * 4 * (kW + 1);                  // one slot's scales
  static constexpr bool kGroups = MODE == kGrouped || MODE == kGated;
  static constexpr int kTokWarps = MODE == kFused ? 4 : 0;               // quantise tokens beside the epilogue's
  static constexpr int kEpiWarps = MODE == kFused ? 4 : MODE == kGated && NT > 64 ? 16 : 8;
  static constexpr int kRoles = MODE == kFused ? 2 : 3;                  // warps that issue: weights, MMAs, tokens
  static constexpr int kThreads = 32 * (kRoles + kTokWarps + kEpiWarps);
  static constexpr int kBox = MODE == kDense ? NT : NT > 64 ? 64 : 16;   // token rows per copy
  static constexpr int kTurn = MODE == kGated ? kEpiWarps * 16 * kTurnRow * 4 : 0;  // epilogue transposes
  static constexpr int kFit = (kSmemMax - kTurn - 2048 - (kGroups ? 4096 : 0)) / kSlot;
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kColsNeeded = kAccs * kW * NT + 2 * kSfCols;
  static constexpr int kCols = kColsNeeded <= 128 ? 128 : kColsNeeded <= 256 ? 256 : 512;
  static_assert(kColsNeeded <= 512, "tensor memory");
  static_assert(kSlot % 1024 == 0, "swizzle atoms");
  static_assert(MODE == kFused || kStages * kSlot >= kSmemMin, "one CTA per SM");
};

struct GemmArgs {
  const uint8_t* wsf;  // weight scale tiles
  const uint8_t* asf;  // token scale tiles
  const float* wts;
  const float* ats;
  int wkb;             // scale tiles along K
  int a_row_tiles;     // pairs: token scale row tiles
  int M, N, C;         // weight rows (of one expert), tokens, chunks of K
  int k_steps;         // MMAs of 64 over the whole of K
  int mt, nt;          // tiles
  int split;           // parts of a tile's K, each a CTA's (1: whole tiles)
  void* y;
  int y_dtype;
  size_t ldy;
  uint32_t* status;
  uint32_t* counters;  // split: arrivals per tile and epilogue warp, zero between calls
  float* part;         // split: [NT][128] sums per CTA
  // grouped: the experts' row segments; tiles are (expert, token tile, m tile)
  const int32_t* offsets;
  const int32_t* counts;
  int E, n_wts;
  // gated: the second (up) matrix, and where the quantised h goes
  const uint8_t* wsf2;
  const float* wts2;
  int n_wts2;
  const float* hts;
  uint8_t* h_codes;
  uint8_t* h_scales;
  int h_kb;
  int early;           // the weights may be read before the preceding kernel ends (grouped: always, and the segments)
  // fused: the tokens
  const void* x;
  int x_dtype;
  size_t ldx;
  int K;
  int stages;          // ring slots (beside them, the tokens of all of K)
  int withhold;        // CTA 0 leaves its first weights' copy unrequested (hq_set_test_fault)
};

// Fused: shared memory of a chunk's tokens, 8 rows: codes (one swizzle atom)
// and scale cells (8 rows x 16 bytes per tile; tcgen05.cp takes 512 bytes, the
// rest is the following tiles' and ends in lanes that no MMA reads).
constexpr int kTokenCodes = 1024;
template <int FMT>
constexpr int kTokenScales = (FMT == HQ_FP4_NV ? 4 : 2) * 128;
template <int FMT>
constexpr size_t token_bytes(int chunks) {
  return static_cast<size_t>(chunks + 1) * kTokenCodes + (static_cast<size_t>(chunks) * kTokenScales<FMT> + 1023) / 1024 * 1024 + 1024;
}

// One item of a CTA's list: a tile and its chunks [c0, c1).
struct Item {
  int m0, n0, n_valid;  // first weight row in its expert, first token row, token rows
  int w_row;            // first weight row in the matrix
  int e;
  int c0, c1;  // chunks of K
};

// A CTA's items.  Expert tiles count token tiles fastest and are dealt out one
// by one, so that the CTAs that take a weight tile's other uses, and an
// expert's tokens' other uses, run at the same time and find them in L2: with
// an even run of tiles per CTA, whose second use of a weight tile comes 6 us
// after the first, the gated product read 427 MB for 340, and the layer took
// 254 us at 4096 tokens (237 with only the second product in runs, 229 so).
// The second product of small token tiles keeps runs: its tiles have few chunks
// and few readers, and the next tile of a run is found sooner (32 tokens 51.0
// us, dealt out 51.7).
template <int NT, int MODE>
struct Walk {
  static constexpr bool kDealt = MODE == kGated || (MODE == kGrouped && NT > 64);
  int u, end;
  const int* first;  // groups: [E + 1] tiles before each expert, then [E] segment starts, [E] row counts
  int e, ni, mi;     // groups: the next tile (dealt out: an expert at or before its own)
  int rows, start;   // groups: of expert e
  __device__ __forceinline__ Walk(const GemmArgs& a, const int* groups) : first(groups) {
    if constexpr (kDealt) {
      u = blockIdx.x;
      end = uniform(first[a.E]);
      e = 0;
    } else if constexpr (MODE == kGrouped) {
      const long all = uniform(first[a.E]);
      u = static_cast<int>(all * blockIdx.x / gridDim.x);
      end = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x);
      e = 0;
      if (u < end) find(a);
    } else {
      u = blockIdx.x / a.split;
      end = a.mt * a.nt;
    }
  }
  // The expert whose tiles include u, first[e] <= u < first[e + 1], from e on,
  // 32 at a time, and u's place in it.
  __device__ __forceinline__ void find(const GemmArgs& a) {
    const int lane = threadIdx.x & 31;
    while (true) {
      const int i = e + 1 + lane;
      const int n = __popc(__ballot_sync(~0u, i < a.E && first[i] <= u));
      e += n;
      if (n < 32) break;
    }
    enter(a);
    const int t = u - uniform(first[e]), nts = (rows + NT - 1) / NT;
    mi = t / nts;
    ni = t - mi * nts;
  }
  __device__ __forceinline__ void enter(const GemmArgs& a) {
    rows = uniform(first[a.E + 1 + a.E + e]);
    start = uniform(first[a.E + 1 + e]);
  }
  // The next item; false at the end.
  __device__ __forceinline__ bool next(const GemmArgs& a, Item& it) {
    if (u >= end) return false;
    it.c0 = 0;
    it.c1 = a.C;
    if constexpr (MODE == kGated || MODE == kGrouped) {
      if constexpr (kDealt) {
        find(a);
        u += gridDim.x;
      } else {
        if (ni * NT >= rows) {
          ni = 0;
          ++mi;
        }
        while (mi >= a.mt || rows == 0) {  // the next expert that has rows
          ++e;
          enter(a);
          ni = mi = 0;
        }
        ++u;
      }
      it.m0 = mi * kM;
      it.n0 = start + ni * NT;
      it.n_valid = min(NT, rows - ni * NT);
      it.w_row = e * a.M + it.m0;
      it.e = e;
      ++ni;
    } else {
      const int tile = u;
      u += gridDim.x;  // parts: one per CTA
      if (a.split > 1) {
        const int part = blockIdx.x - tile * a.split;
        it.c0 = a.C * part / a.split;
        it.c1 = a.C * (part + 1) / a.split;
      }
      // token tiles fastest: CTAs that run together share weight tiles in L2
      const int mi_ = tile / a.nt, ni_ = tile - mi_ * a.nt;
      it.m0 = mi_ * kM;
      it.n0 = ni_ * NT;
      it.n_valid = min(NT, a.N - it.n0);
      it.w_row = it.m0;
      it.e = 0;
    }
    return true;
  }
};

// The experts' tiles and segments into shared memory, by the whole CTA, a scan
// over all threads (one warp's took 0.7 us for 256 experts, before the first
// copy).  start, count: those of expert threadIdx.x.
template <int NT, int THREADS>
__device__ __forceinline__ void load_groups(const GemmArgs& a, int* first, int start, int count) {
  __shared__ int sums[THREADS / 32];
  int* starts = first + a.E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int e0 = 0; e0 < a.E; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    if (e0 > 0 && e < a.E) {
      start = __ldg(a.offsets + e);
      count = __ldg(a.counts + e);
    }
    const int n = e < a.E ? (count + NT - 1) / NT * a.mt : 0;
    int s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, s, o);
      if (lane >= o) s += v;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      before += w < warp ? sums[w] : 0;
      carry += sums[w];
    }
    if (e < a.E) {
      first[e] = before + s - n;
      starts[e] = start;
      starts[a.E + e] = count;
      if (e == a.E - 1) first[a.E] = before + s;
    }
    __syncthreads();
  }
}

// The two tensor scales of a product (nullptr: 1).  As one factor where their
// product is a normal number (or one of them is 0); else one after the other,
// the larger first, so that a result within fp32's range is not lost to a
// product of scales that is infinite or has no bits left.
struct Alpha {
  float first, second;
  __device__ __forceinline__ Alpha(float w, float t) {
    const float p = fabsf(__fmul_rn(w, t));
    const bool one = (p >= 0x1p-126f && p < INFINITY) || w == 0.f || t == 0.f;
    const bool swap = fabsf(w) < fabsf(t);
    first = one ? __fmul_rn(w, t) : swap ? t : w;
    second = one ? 1.f : swap ? w : t;
  }
  __device__ __forceinline__ float operator()(float sum) const { return sum * first * second; }
};
__device__ __forceinline__ float scale_of(const float* p, int i) { return p != nullptr ? __ldg(p + i) : 1.f; }

// Rows y[0 .. n) of one column from P columns of a lane's accumulator.
template <int P, typename T>
__device__ __forceinline__ void store_column(T* y, size_t ldy, const float (&f)[P], int n) {
  if (n >= P) {
#pragma unroll
    for (int j = 0; j < P; ++j, y += ldy) *y = from_f32<T>(f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < P; ++j, y += ldy) {
      if (j < n) *y = from_f32<T>(f[j]);
    }
  }
}

template <int P>
__device__ __forceinline__ void store_any(const GemmArgs& a, size_t row, int m, const float (&f)[P], int n) {
  const size_t o = row * a.ldy + m;
  if (a.y_dtype == HQ_BF16) store_column<P>(static_cast<__nv_bfloat16*>(a.y) + o, a.ldy, f, n);
  else if (a.y_dtype == HQ_F16) store_column<P>(static_cast<__half*>(a.y) + o, a.ldy, f, n);
  else store_column<P>(static_cast<float*>(a.y) + o, a.ldy, f, n);
}

// 16 values of token `row` from `col` on (0 outside).
__device__ __forceinline__ void load_token(const GemmArgs& a, int row, int col, float (&v)[16]) {
  if (row < a.N && col < a.K) {
    const size_t o = row * a.ldx + col;
    if (a.x_dtype == HQ_BF16) load_chunk<__nv_bfloat16, 16>(static_cast<const __nv_bfloat16*>(a.x) + o, v);
    else if (a.x_dtype == HQ_F16) load_chunk<__half, 16>(static_cast<const __half*>(a.x) + o, v);
    else load_chunk<float, 16>(static_cast<const float*>(a.x) + o, v);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
  }
}

// P (16 or 32) accumulator columns from c on.
template <int P>
__device__ __forceinline__ void load_columns(uint32_t d, float (&f)[P]) {
  uint32_t v[P / 16][16];
#pragma unroll
  for (int i = 0; i < P / 16; ++i) tc::tc_ld16(d + 16 * i, v[i]);
  tc::tc_wait_ld();
#pragma unroll
  for (int i = 0; i < P / 16; ++i) {
    tc::tc_tie16(v[i]);
#pragma unroll
    for (int j = 0; j < 16; ++j) f[16 * i + j] = __uint_as_float(v[i][j]);
  }
}

// ------------------------------------------------------------------ kernel

template <int FMT, int NT, int MODE>
__global__ void __launch_bounds__(Shape<FMT, NT, MODE>::kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap wmap2,
                const __grid_constant__ CUtensorMap amap, const GemmArgs a) {
  using S = Shape<FMT, NT, MODE>;
  constexpr bool GROUPED = S::kGroups;
  constexpr bool FUSED = MODE == kFused;
  const int ST = FUSED ? a.stages : S::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float* turn_buf = reinterpret_cast<float*>(ring + ST * S::kSlot);
  uint8_t* tok = ring + ST * S::kSlot;  // fused: the tokens' codes, then their scales
  uint8_t* tok_sf = tok + (a.C + 1) * kTokenCodes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ST * S::kSlot +
                                               (FUSED ? token_bytes<FMT>(a.C) : static_cast<size_t>(S::kTurn)));
  uint64_t* empty = full + ST;
  uint64_t* dfull = empty + ST;
  uint64_t* dempty = dfull + S::kAccs;
  uint64_t* tok_full = dempty + S::kAccs;
  uint64_t* drain = tok_full + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  __shared__ int first[GROUPED ? 3 * kMaxGroups + 1 : 1];
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  int start = 0, count = 0;
  if (GROUPED && threadIdx.x < a.E) {  // always early: see GemmArgs
    start = __ldg(a.offsets + threadIdx.x);
    count = __ldg(a.counts + threadIdx.x);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + i, S::kRoles - 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < S::kAccs; ++i) {
      mbar_init(dfull + i, 1);
      mbar_init(dempty + i, S::kEpiWarps);
    }
    mbar_init(tok_full, S::kTokWarps + S::kEpiWarps);
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&wmap);
    if (MODE == kGated) prefetch_tensormap(&wmap2);
    if (!FUSED) prefetch_tensormap(&amap);
  }
  if (warp == 1) {
    tc::tmem_alloc(tslot, S::kCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t sf_cols = tmem + S::kAccs * S::kW * NT;
  if constexpr (GROUPED) load_groups<NT, S::kThreads>(a, first, start, count);
  bool ok = true;

  if (warp == 0) {
    if (a.early == 0) pdl_wait();
    if (FUSED) pdl_launch_dependents();
    Walk<NT, MODE> w(a, first);
    Item it;
    int slot = 0, turn = 0, n = 0;
    while (ok && w.next(a, it)) {
      for (int c = it.c0; c < it.c1; ++c) {
        if (n >= ST && !warp_wait(empty + slot, turn ^ 1)) {
          ok = false;
          break;
        }
        const int bytes = min(S::kTiles, a.wkb - c * S::kTiles) * 512;
        uint8_t* p = ring + slot * S::kSlot;
        const size_t sf = (static_cast<size_t>(it.w_row >> 7) * a.wkb + c * S::kTiles) * 512;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + slot, S::kW * (kWBytes + bytes));
          if (a.withhold == 0 || blockIdx.x != 0 || n != 0) tma_load_2d(p, &wmap, c * (kChunk / 2), it.w_row, full + slot);
          bulk_g2s(p + S::kSfOff, a.wsf + sf, bytes, full + slot);
          if constexpr (MODE == kGated) {
            tma_load_2d(p + kWBytes, &wmap2, c * (kChunk / 2), it.w_row, full + slot);
            bulk_g2s(p + S::kSfOff + S::kSf, a.wsf2 + sf, bytes, full + slot);
          }
        }
        ++n;
        if (++slot == ST) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    ok = drain_slots(full, ST, n) && ok;
  } else if (!FUSED && warp == 2) {
    Walk<NT, MODE> w(a, first);
    pdl_wait();
    // After the wait, so that whatever precedes this kernel is complete when
    // the next one starts.
    pdl_launch_dependents();
    Item it;
    int slot = 0, turn = 0, n = 0;
    while (ok && w.next(a, it)) {
      const int boxes = (min(it.n_valid, NT) + S::kBox - 1) / S::kBox;
      for (int c = it.c0; c < it.c1; ++c) {
        if (n >= ST && !warp_wait(empty + slot, turn ^ 1)) {
          ok = false;
          break;
        }
        const int bytes = min(S::kTiles, a.wkb - c * S::kTiles) * 512;
        uint8_t* p = ring + slot * S::kSlot + S::kW * kWBytes;
        uint8_t* psf = ring + slot * S::kSlot + S::kSfOff + S::kW * S::kSf;
        const uint8_t* sf = a.asf + (static_cast<size_t>(it.n0 >> 7) * a.wkb + c * S::kTiles) * 512;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + slot, boxes * S::kBox * 128 + bytes);
          for (int i = 0; i < boxes; ++i) {
            tma_load_2d(p + i * S::kBox * 128, &amap, c * (kChunk / 2), it.n0 + i * S::kBox, full + slot);
          }
          bulk_g2s(psf, sf, bytes, full + slot);
        }
        ++n;
        if (++slot == ST) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    ok = drain_slots(full, ST, n) && ok;
  } else if (warp == 1) {
    const uint32_t d0 = uniform(tmem), sf0 = uniform(sf_cols), ring0 = uniform(smem_u32(ring));
    Walk<NT, MODE> w(a, first);
    Item it;
    int slot = 0, par = 0, acc = 0, accn = 0, n = 0;
    if (FUSED) ok = warp_wait(tok_full, 0);
    const uint32_t tok0 = uniform(smem_u32(tok)), tok_sf0 = uniform(smem_u32(tok_sf));
    while (ok && w.next(a, it)) {
      const uint32_t d = d0 + acc * S::kW * NT;
      if (accn >= S::kAccs && !warp_wait(dempty + acc, (accn / S::kAccs - 1) & 1)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const int n_mma = (it.n_valid + 15) / 16 * 16;
      // the tokens' rows within their scale tile: 0 or 64 (two columns)
      const uint32_t half = NT < 128 ? ((it.n0 & 127) >> 5) : 0;
      for (int c = it.c0; c < it.c1; ++c) {
        if (!warp_wait(full + slot, par)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t p = ring0 + slot * S::kSlot;
        const uint32_t sfa = sf0 + (n & 1) * S::kSfCols, sfb = sfa + S::kW * S::kTiles * 4, sp = p + S::kSfOff;
        const uint64_t da = desc_sw128(p), db = desc_sw128(FUSED ? tok0 + c * kTokenCodes : p + S::kW * kWBytes);
        const uint32_t sp_tok = FUSED ? tok_sf0 + c * kTokenScales<FMT> : sp + S::kW * S::kSf;
        const int steps = min(4, a.k_steps - 4 * c);
        const uint32_t first_sum = c > it.c0 ? 1u : 0u;
        ++n;
        if (elect_one()) {
#pragma unroll
          for (int t = 0; t < S::kTiles; ++t) {
#pragma unroll
            for (int i = 0; i < S::kW; ++i) tc_copy_scales(sfa + 4 * (i * S::kTiles + t), sp + i * S::kSf + 512 * t);
            tc_copy_scales(sfb + 4 * t, sp_tok + (FUSED ? 128 : 512) * t);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s < steps) {
#pragma unroll
              for (int i = 0; i < S::kW; ++i) {
                const int t = FMT == HQ_FP4_NV ? s : s >> 1, id = FMT == HQ_FP4_NV ? 0 : 2 * (s & 1);
                tc_mma_scaled<FMT>(d + i * NT, da + i * (kWBytes >> 4) + 2 * s, db + 2 * s, idesc_fp4(FMT, n_mma, id),
                                   sfa + 4 * (i * S::kTiles + t), sfb + 4 * t + half,
                                   s > 0 ? 1u : first_sum);
              }
            }
          }
          tc::tc_commit(empty + slot);
          if (c + 1 == it.c1) tc::tc_commit(dfull + acc);
        }
        if (++slot == ST) {
          slot = 0;
          par ^= 1;
        }
      }
      ++accn;
      acc = accn % S::kAccs;
    }
    // no MMA may be in flight when tensor memory is freed
    if (elect_one()) tc::tc_commit(drain);
    ok = warp_wait(drain, 0) && ok;
  } else {
    pdl_wait();
    if constexpr (FUSED) {
      // All of the tokens, once per CTA, while the first weights are on their
      // way: a thread takes 16 values, two loads ahead of each other.
      constexpr int kWorkers = 32 * (S::kTokWarps + S::kEpiWarps);
      const SixTs ts(a.ats);
      const int per_row = a.C * (kChunk / 16);
      struct At {
        int row, b;  // 16-value piece b of a row
      };
      auto step = [&](At& t) {
        t.b += kWorkers;
        while (t.b >= per_row) {
          t.b -= per_row;
          ++t.row;
        }
      };
      auto pack = [&](const At& t, float (&v)[16]) {  // all lanes; rows and workers are multiples of 16 pieces
        const Packed16 q = pack16<FMT>(v, top_of(v), ts, 1);
        if (t.row >= a.N) return;
        const int c = t.b >> 4, blk = t.b & 15;
        // 128 bytes a row, 16-byte pieces exchanged by the row's place in its group of 8
        *reinterpret_cast<uint2*>(tok + c * kTokenCodes + t.row * 128 + (((blk >> 1) ^ t.row) << 4) + (blk & 1) * 8) = q.codes;
        constexpr int kPer = FMT == HQ_FP4_NV ? 1 : 2;  // threads per block
        tok_sf[c * kTokenScales<FMT> + blk / (4 * kPer) * 128 + t.row * 16 + (blk / kPer & 3)] = static_cast<uint8_t>(q.byte);
      };
      At t0{0, static_cast<int>(threadIdx.x) - 32 * S::kRoles - kWorkers}, t1;
      float v0[16], v1[16];
      step(t0);
      load_token(a, t0.row, t0.b * 16, v0);
      while (__any_sync(~0u, t0.row < a.N)) {
        t1 = t0;
        step(t1);
        load_token(a, t1.row, t1.b * 16, v1);
        pack(t0, v0);
        t0 = t1;
        step(t0);
        load_token(a, t0.row, t0.b * 16, v0);
        pack(t1, v1);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tok_full);
    }
    if (warp >= S::kRoles + S::kTokWarps) {
      const int ew = warp - S::kRoles - S::kTokWarps, quarter = warp & 3;
      constexpr int kParts = S::kEpiWarps / 4;  // warps that share a lane quarter split the columns
      const int col0 = (ew >> 2) * (NT / kParts), col1 = col0 + NT / kParts;
      const int mrow = quarter * 32 + lane;
      const SixTs hts(MODE == kGated ? a.hts : nullptr);
      const float ats = scale_of(a.ats, 0);
      Walk<NT, MODE> w(a, first);
      Item it;
      int acc = 0, accn = 0;
      while (ok && w.next(a, it)) {
        // before the wait, which hides the loads
        const Alpha alpha(scale_of(a.wts, a.n_wts > 1 ? it.e : 0), ats);
        const Alpha alpha2(MODE == kGated ? scale_of(a.wts2, a.n_wts2 > 1 ? it.e : 0) : 1.f, ats);
        if (!warp_wait(dfull + acc, (accn / S::kAccs) & 1)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t d = tmem + acc * S::kW * NT + (static_cast<uint32_t>(quarter * 32) << 16);
        const bool whole = it.c0 == 0 && it.c1 == a.C;
        const int m = it.m0 + mrow;
        if constexpr (MODE == kGated) {
          // 16 tokens at a time: h of this lane's feature, a transpose through
          // shared memory, then 16 features of one token per lane
          float* buf = turn_buf + ew * 16 * kTurnRow;
          // All of the warp's columns first, so that the next tile's MMAs can have
          // the accumulators while h is computed and packed.
          constexpr int kCols = NT / kParts;
          float g[kCols], u[kCols];
          if (col0 < it.n_valid) {
            load_columns<kCols>(d + col0, g);
            load_columns<kCols>(d + NT + col0, u);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dempty + acc);
#pragma unroll
          for (int c1 = 0; c1 < kCols; c1 += 16) {
            const int c = col0 + c1;
            if (c >= it.n_valid) break;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (c + i >= it.n_valid) break;
              const float x = alpha(g[c1 + i]);
              // expf and an IEEE division, as in hq_moe_experts: the fast ones are off by up to
              // 2 + 1.2 |g| ulps, enough to move h across a border between two codes.
              buf[i * kTurnRow + lane] = x / (1.f + expf(-x)) * alpha2(u[c1 + i]);
            }
            __syncwarp();
            const int token = lane & 15, part = lane >> 4;
            // (Rows without a token hold anything: as zeros they keep the warp from the
            // quantiser's division, 32 tokens 51.2 us instead of 54.9.)
            const bool there = c + token < it.n_valid;
            float v[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
              if (there) f = *reinterpret_cast<const float4*>(buf + token * kTurnRow + part * 16 + 4 * i);
              v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
            }
            const Packed16 p = pack16<FMT>(v, top_of(v), hts, 16);
            const uint32_t other = __shfl_xor_sync(~0u, p.byte, 16);
            if (there) {
              const long row = it.n0 + c + token;
              const int f0 = it.m0 + quarter * 32;  // the warp's first feature
              *reinterpret_cast<uint2*>(a.h_codes + row * (a.M / 2) + (f0 + part * 16) / 2) = p.codes;
              if (part == 0) {
                if constexpr (FMT == HQ_FP4_NV) {
                  uint8_t* s = a.h_scales + scale_cell(row, f0 >> 6, a.h_kb) + (quarter & 1) * 2;
                  *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(p.byte | other << 8);
                } else {
                  a.h_scales[scale_cell(row, f0 >> 7, a.h_kb) + quarter] = static_cast<uint8_t>(p.byte);
                }
              }
            }
            __syncwarp();
          }
        } else if (whole) {
          constexpr int P = NT / kParts < 32 ? 16 : 32;
          for (int c = col0; c < col1 && c < it.n_valid; c += P) {
            float f[P];
            load_columns<P>(d + c, f);
            if (m < a.M) {
#pragma unroll
              for (int j = 0; j < P; ++j) f[j] = alpha(f[j]);
              store_any<P>(a, it.n0 + c, m, f, it.n_valid - c);
            }
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dempty + acc);
        } else if constexpr (!GROUPED) {
          const int tile = blockIdx.x / a.split;
          constexpr size_t kPart = static_cast<size_t>(NT) * kM;
          float* mine = a.part + blockIdx.x * kPart;
          for (int c = col0; c < col1 && c < it.n_valid; c += 16) {
            float f[16];
            load_columns<16>(d + c, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(mine + (c + i) * kM + mrow, f[i]);
          }
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dempty + acc);
          // Each warp's share of the tile is counted on its own: the last of the
          // tile's CTAs to bring it adds the parts, in their order.
          uint32_t last = 0;
          uint32_t* counter = a.counters + tile * kMaxEpiWarps + ew;
          if (lane == 0 && col0 < it.n_valid) {
            __threadfence();
            last = atomicAdd(counter, 1u) == static_cast<uint32_t>(a.split - 1) ? 1u : 0u;
          }
          if (__shfl_sync(~0u, last, 0) != 0) {
            __threadfence();
            if (lane == 0) *counter = 0;
            for (int c = col0; c < col1 && c < it.n_valid; c += 16) {
              float f[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) f[j] = 0.f;
              for (int i = 0; i < a.split; ++i) {  // 16 loads in flight
                const float* p = a.part + (static_cast<size_t>(tile) * a.split + i) * kPart + c * kM + mrow;
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __ldcg(p + j * kM);
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] += v[j];
              }
              if (m < a.M) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = alpha(f[j]);
                store_any<16>(a, it.n0 + c, m, f, it.n_valid - c);
              }
            }
          }
        }
        ++accn;
        acc = accn % S::kAccs;
      }
    }
  }
  if (!ok) record_error(a.status, HQ_DEV_TIMEOUT);
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, S::kCols);
}

// ------------------------------------------------------------------ pairs
//
// Large products: two CTAs of a cluster on one tile of 256 weight rows x 256
// tokens (cta_group::2).  Each brings its own 128 weight rows and half of the
// tokens, and the tensor cores of both read both halves, so a chunk costs each
// SM 36 KB of copies and 32 KB of operand reads instead of 54 and 48: a single
// CTA's 128 x 256 tile is bound by shared-memory bandwidth (about 108 KB a
// chunk, 843 cycles at 128 bytes a cycle, for 512 cycles of MMAs).
//
// The even CTA's MMA warp issues for both.  It waits for its own slot and for
// the odd CTA's, whose warp 1 passes its slots' arrivals on; commits free the
// slots and hand over the accumulators in both CTAs.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrive on CTA 0's barrier at the address of this CTA's `bar`.  What the
// arrivals pass on is not plain memory: copies that have landed in shared
// memory (their completion, which is a release at cluster scope, was waited for,
// and nothing is cached between it and the MMAs), accumulators that have been
// read (tcgen05 fences order those).  So neither side releases or acquires at
// cluster scope; with it the product at 8192 x 8192 x 4096 took 170 us instead
// of 97.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint32_t smem) {
  const uint64_t desc = tc::smem_desc(smem, 0, 128);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <int FMT>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
  if constexpr (FMT == HQ_FP4_NV) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  }
}

template <int FMT>
struct PairShape {
  static constexpr int NT = 256;
  static constexpr int kTiles = kChunk / (FMT == HQ_FP4_NV ? 64 : 128);
  static constexpr int kSf = kTiles * 512;
  static constexpr int kABytes = NT / 2 * kChunk / 2;
  static constexpr int kSfOff = kWBytes + kABytes;
  static constexpr int kSlot = (kSfOff + 3 * kSf + 1023) / 1024 * 1024;
  static constexpr int kStages = (kSmemMax - 2048) / kSlot;
  static constexpr int kSfCols = kTiles * 4 * 3;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (3 + kEpiWarps);
  static_assert(NT + 2 * kSfCols <= 512, "tensor memory");
  static_assert(kStages * kSlot >= kSmemMin, "one CTA per SM");
};

template <int FMT>
__global__ void __launch_bounds__(PairShape<FMT>::kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap, const GemmArgs a) {
  using S = PairShape<FMT>;
  constexpr int NT = S::NT, ST = S::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + ST * S::kSlot);
  uint64_t* peer = full + ST;  // CTA 0: the other CTA's slot is full
  uint64_t* empty = peer + ST;
  uint64_t* dfull = empty + ST;
  uint64_t* dempty = dfull + 1;
  uint64_t* drain = dempty + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rank = uniform(static_cast<int>(cluster_rank()));
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1, tiles = a.mt * a.nt;
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(full + i, 2);
      mbar_init(peer + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(dfull, 1);
    mbar_init(dempty, 2 * S::kEpiWarps);
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&amap);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *tslot, sf_cols = tmem + NT;
  bool ok = true;

  if (warp == 0) {
    if (a.early == 0) pdl_wait();
    int slot = 0, turn = 0, n = 0;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const int row = t / a.nt * 256 + rank * kM;
      for (int c = 0; c < a.C; ++c) {
        if (n >= ST && !warp_wait(empty + slot, turn ^ 1)) {
          ok = false;
          break;
        }
        // an odd number of row tiles: the last pair's second CTA has no weights
        // (its copies read zeros past the last row) and no scales
        const int bytes = row < a.M ? min(S::kTiles, a.wkb - c * S::kTiles) * 512 : 0;
        uint8_t* p = ring + slot * S::kSlot;
        const uint8_t* sf = a.wsf + (static_cast<size_t>(row >> 7) * a.wkb + c * S::kTiles) * 512;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + slot, kWBytes + bytes);
          if (a.withhold == 0 || blockIdx.x != 0 || n != 0) tma_load_2d(p, &wmap, c * (kChunk / 2), row, full + slot);
          if (bytes > 0) bulk_g2s(p + S::kSfOff, sf, bytes, full + slot);
        }
        ++n;
        if (++slot == ST) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    ok = drain_slots(full, ST, n) && ok;
  } else if (warp == 2) {
    pdl_wait();
    pdl_launch_dependents();  // after the wait, as in gemm_kernel
    int slot = 0, turn = 0, n = 0;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const int n0 = t % a.nt * NT;
      const int row_tiles = min(2, a.a_row_tiles - (n0 >> 7));
      for (int c = 0; c < a.C; ++c) {
        if (n >= ST && !warp_wait(empty + slot, turn ^ 1)) {
          ok = false;
          break;
        }
        const int bytes = min(S::kTiles, a.wkb - c * S::kTiles) * 512;
        uint8_t* p = ring + slot * S::kSlot;
        const uint8_t* sf = a.asf + (static_cast<size_t>(n0 >> 7) * a.wkb + c * S::kTiles) * 512;
        const size_t next = static_cast<size_t>(a.wkb) * 512;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + slot, S::kABytes + row_tiles * bytes);
          tma_load_2d(p + kWBytes, &amap, c * (kChunk / 2), n0 + rank * (NT / 2), full + slot);
          bulk_g2s(p + S::kSfOff + S::kSf, sf, bytes, full + slot);
          if (row_tiles > 1) bulk_g2s(p + S::kSfOff + 2 * S::kSf, sf + next, bytes, full + slot);
        }
        ++n;
        if (++slot == ST) {
          slot = 0;
          turn ^= 1;
        }
      }
    }
    ok = drain_slots(full, ST, n) && ok;
  } else if (warp == 1 && rank != 0) {
    int slot = 0, par = 0;
    for (int t = pair; ok && t < tiles; t += pairs) {
      for (int c = 0; c < a.C; ++c) {
        if (!warp_wait(full + slot, par)) {
          ok = false;
          break;
        }
        if (elect_one()) arrive_leader(peer + slot);
        if (++slot == ST) {
          slot = 0;
          par ^= 1;
        }
      }
    }
    ok = warp_wait(drain, 0) && ok;  // the leader's MMAs read this CTA's slots
  } else if (warp == 1) {
    const uint32_t d = uniform(tmem), sf0 = uniform(sf_cols), ring0 = uniform(smem_u32(ring));
    int slot = 0, par = 0, n = 0, tile = 0;
    // M = 256
    constexpr uint32_t kIdesc = idesc_fp4(FMT, NT, 0) - (static_cast<uint32_t>(kM >> 4) << 24) + (16u << 24);
    for (int t = pair; ok && t < tiles; t += pairs, ++tile) {
      if (tile > 0 && !warp_wait(dempty, (tile - 1) & 1)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      for (int c = 0; c < a.C; ++c) {
        if (!warp_wait(full + slot, par) || !warp_wait(peer + slot, par)) {
          ok = false;
          break;
        }
        tc::tc_fence_after();
        const uint32_t p = ring0 + slot * S::kSlot;
        const uint32_t sfa = sf0 + (n & 1) * S::kSfCols, sfb = sfa + S::kTiles * 4, sp = p + S::kSfOff;
        const uint64_t da = desc_sw128(p), db = desc_sw128(p + kWBytes);
        const int steps = min(4, a.k_steps - 4 * c);
        const uint32_t first_sum = c > 0 ? 1u : 0u;
        ++n;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < S::kTiles; ++i) {
            pair_copy_scales(sfa + 4 * i, sp + 512 * i);
            pair_copy_scales(sfb + 8 * i, sp + S::kSf + 512 * i);
            pair_copy_scales(sfb + 8 * i + 4, sp + 2 * S::kSf + 512 * i);
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s < steps) {
              const int i = FMT == HQ_FP4_NV ? s : s >> 1;
              const uint32_t id = FMT == HQ_FP4_NV ? 0u : 2u * (s & 1);
              pair_mma<FMT>(d, da + 2 * s, db + 2 * s, kIdesc | id << 29 | id << 4, sfa + 4 * i, sfb + 8 * i,
                            s > 0 ? 1u : first_sum);
            }
          }
          pair_commit(empty + slot);
          if (c + 1 == a.C) pair_commit(dfull);
        }
        if (++slot == ST) {
          slot = 0;
          par ^= 1;
        }
      }
    }
    // no MMA may be in flight when tensor memory is freed, in either CTA
    if (elect_one()) pair_commit(drain);
    ok = warp_wait(drain, 0) && ok;
  } else {
    pdl_wait();
    const int ew = warp - 3, quarter = warp & 3;
    const int col0 = (ew >> 2) * (NT / 2), col1 = col0 + NT / 2;
    const int mrow = quarter * 32 + lane;
    const Alpha alpha(scale_of(a.wts, 0), scale_of(a.ats, 0));
    const uint32_t d = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int tile = 0;
    for (int t = pair; ok && t < tiles; t += pairs, ++tile) {
      if (!warp_wait(dfull, tile & 1)) {
        ok = false;
        break;
      }
      tc::tc_fence_after();
      const int n0 = t % a.nt * NT, n_valid = min(NT, a.N - n0);
      const int m = t / a.nt * 256 + rank * kM + mrow;
      for (int c = col0; c < col1 && c < n_valid; c += 32) {
        float f[32];
        load_columns<32>(d + c, f);
        if (c + 32 >= min(col1, n_valid)) {  // the warp's last: the accumulators are read
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(dempty);
        }
        if (m < a.M) {
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = alpha(f[j]);
          store_any<32>(a, n0 + c, m, f, n_valid - c);
        }
      }
      if (col0 >= n_valid) {
        __syncwarp();
        if (lane == 0) arrive_leader(dempty);
      }
    }
  }
  if (!ok) record_error(a.status, HQ_DEV_TIMEOUT);
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();  // no arrival or operand read of the other CTA is left
  if (warp == 1) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// ------------------------------------------------------------------ host

constexpr size_t kStatusBytes = 256;
constexpr size_t kCounterBytes = 8192;  // a word per epilogue warp and CTA of a split grid
constexpr int kMaxGrid = static_cast<int>(kCounterBytes / 4 / kMaxEpiWarps);
static_assert(kStatusBytes + kCounterBytes == 8448, "what callers zero, in hq.h and the Python layers");

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// How a dense product runs.
struct Plan {
  int nt_size;  // tokens per tile
  bool pair;    // tiles of 256 x 256, two CTAs each
  int mt, nt, C, grid, split;
};

// Parts of a tile's K are worth their exchange from about 8 chunks each on, for
// more than 32 tokens from 16 and three parts.  2048 x 8192: 16 tokens 9.4 us
// in 4 parts, 10.4 in 2, 10.8 in 9, 11.9 whole; 128 tokens 14.5 us in 4 parts,
// 18.9 in 9, 14.0 whole.  2048 x 16384 at 128 tokens: 17.2 us in 4 parts, 19.5
// in 2, 21.6 in 9, 23.4 whole.  8192 x 8192 at 64: 15.6 us in 2 parts, 13.3
// whole.  (An even split of 96 tiles over all 148 CTAs, 12288 x 4096 at 16, was
// slower too when it was tried: 11.6 us against 8.9 whole.)
int parts_of(long tiles, long sms, int nt_size, int C) {
  const long s = std::min<long>(sms / tiles, C / (nt_size <= 32 ? 8 : 16));
  return static_cast<int>(s < (nt_size <= 32 ? 2 : 3) ? 1 : s);
}

Plan plan_of(int M, int N, int K) {
  Plan p{};
  const long sms = std::min(sm_count(), kMaxGrid);
  p.C = (K + kChunk - 1) / kChunk;
  p.mt = (M + kM - 1) / kM;
  p.nt_size = N <= 32 ? 32 : N <= 64 ? 64 : 128;
  p.nt = (N + p.nt_size - 1) / p.nt_size;
  const long tiles = static_cast<long>(p.mt) * p.nt;
  // More than one wave of 128 x 128 tiles: pairs.  4100 x 4128 at 333 tokens
  // (99 tiles) 11.8 us, in pairs 13.5; 12288 x 4096 at 200 (192 tiles) 15.3 us,
  // in pairs 12.9; 8192 x 8192 at 4096 162 us, in pairs 115 (at full clock).
  if (N > 128 && tiles > sms) {
    p.pair = true;
    p.nt_size = 256;
    p.mt = (M + 255) / 256;
    p.nt = (N + 255) / 256;
    p.grid = static_cast<int>(std::min(sms / 2, static_cast<long>(p.mt) * p.nt) * 2);
    return p;
  }
  p.split = parts_of(tiles, sms, p.nt_size, p.C);
  p.grid = static_cast<int>(std::min(sms, tiles * p.split));
  return p;
}

// Room for every plan of up to N tokens: a workspace for N serves all smaller
// batches too.
size_t part_bound(int N, int K) {
  const int nt = N <= 32 ? 32 : N <= 64 ? 64 : 128;
  return (K + kChunk - 1) / kChunk < 16
             ? 0
             : static_cast<size_t>(std::min(sm_count(), kMaxGrid)) * nt * kM * sizeof(float);
}

template <int FMT, int NT, int MODE>
cudaError_t gemm_launch(const CUtensorMap& wmap, const CUtensorMap& wmap2, const CUtensorMap& amap,
                        const GemmArgs& a, int grid, cudaStream_t st) {
  using S = Shape<FMT, NT, MODE>;
  const size_t smem = 1024 + static_cast<size_t>(S::kStages) * S::kSlot + S::kTurn + 512;
  return launch_pdl(gemm_kernel<FMT, NT, MODE>, dim3(grid), dim3(S::kThreads), smem, st, true, wmap, wmap2, amap,
                    a);
}

// Ring slots of a fused launch beside the tokens of C chunks (0: no room).
template <int FMT>
int fused_stages(int C) {
  using S = Shape<FMT, 32, kFused>;
  const long room = kSmemMax - 2048 - static_cast<long>(token_bytes<FMT>(C));
  const long n = room / S::kSlot;
  return n < 4 ? 0 : static_cast<int>(std::min<long>(n, 8));
}
// One launch or two: every CTA quantises all of the tokens, about 1.7 us per
// 8192 values, a kernel of its own costs about 2.5 us.  28672 x 8192: one token
// 25.5 us against 26.5, two 28.2 against 26.3, eight 38.3 against 26.8; 4096 x
// 4096: one 7.9 against 8.9, two 8.1 against 8.8, eight 11.9 against 8.8.
// 12288 values are about even: one token of 4096 x 12288 11.8 against 12.2, of
// 12288 x 12288 19.4 against 19.3, of 28672 x 12288 37.7 against 36.9.
bool fused_fits(int fmt, int N, int K) {
  const int C = (K + kChunk - 1) / kChunk;
  return N <= kFusedTokens && static_cast<long>(N) * K <= 8192 &&
         (fmt == HQ_FP4_NV ? fused_stages<HQ_FP4_NV>(C) : fused_stages<HQ_FP4_MX>(C)) > 0;
}

template <int FMT>
cudaError_t fused_launch(const CUtensorMap& wmap, GemmArgs& a, int grid, cudaStream_t st) {
  using S = Shape<FMT, 32, kFused>;
  a.stages = fused_stages<FMT>(a.C);
  const size_t smem = std::max<size_t>(
      kSmemMin, 1024 + static_cast<size_t>(a.stages) * S::kSlot + token_bytes<FMT>(a.C) + 512);
  return launch_pdl(gemm_kernel<FMT, 32, kFused>, dim3(grid), dim3(S::kThreads), smem, st, true, wmap, wmap, wmap, a);
}

template <int FMT>
cudaError_t pair_launch(const CUtensorMap& wmap, const CUtensorMap& amap, const GemmArgs& a, int grid,
                        cudaStream_t st) {
  using S = PairShape<FMT>;
  const size_t smem = 1024 + static_cast<size_t>(S::kStages) * S::kSlot + 512;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(pair_kernel<FMT>), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  note_launch();
  return cudaLaunchKernelEx(&cfg, pair_kernel<FMT>, wmap, amap, a);
}

template <int FMT>
cudaError_t dense_launch(int nt, const CUtensorMap& wmap, const CUtensorMap& amap, const GemmArgs& a, int grid,
                         cudaStream_t st) {
  switch (nt) {
    case 32: return gemm_launch<FMT, 32, kDense>(wmap, wmap, amap, a, grid, st);
    case 64: return gemm_launch<FMT, 64, kDense>(wmap, wmap, amap, a, grid, st);
    default: return gemm_launch<FMT, 128, kDense>(wmap, wmap, amap, a, grid, st);
  }
}

template <int FMT, int MODE>
cudaError_t group_launch(int nt, const CUtensorMap& wmap, const CUtensorMap& wmap2, const CUtensorMap& amap,
                         const GemmArgs& a, int grid, cudaStream_t st) {
  return nt == 64 ? gemm_launch<FMT, 64, MODE>(wmap, wmap2, amap, a, grid, st)
                  : gemm_launch<FMT, 128, MODE>(wmap, wmap2, amap, a, grid, st);
}

cudaError_t code_map(CUtensorMap* map, const uint8_t* codes, long rows, int K, int box_rows) {
  return tensor_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, static_cast<uint64_t>(K / 2),
                       static_cast<uint64_t>(rows), static_cast<uint64_t>(K / 2), kChunk / 2, box_rows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
}

// What a dense product's launch takes from its weights and plan.
GemmArgs dense_args(const hq_fp4_matrix* w, const Plan& p, int N, void* y, hq_dtype yd, size_t ldy, uint8_t* ws,
                    uint8_t* part) {
  GemmArgs a{};
  a.wsf = w->scales;
  a.wts = w->tensor_scale;
  a.n_wts = 1;
  a.wkb = scale_tiles(w->format, w->K);
  a.a_row_tiles = (N + 127) / 128;
  a.M = w->rows;
  a.N = N;
  a.C = p.C;
  a.k_steps = (w->K + 63) / 64;
  a.mt = p.mt;
  a.nt = p.nt;
  a.split = p.split;
  a.y = y;
  a.y_dtype = yd;
  a.ldy = ldy;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kStatusBytes);
  a.part = reinterpret_cast<float*>(part);
  a.withhold = take_test_fault() ? 1 : 0;
  return a;
}

// y = W q(x) for a few tokens in one launch.
cudaError_t launch_fused(const hq_fp4_matrix* w, const void* x, hq_dtype xd, size_t ldx, int N, const float* x_scale,
                         void* y, hq_dtype yd, size_t ldy, uint8_t* ws, uint8_t* part, cudaStream_t st) {
  const Plan p = plan_of(w->rows, N, w->K);
  CUtensorMap wmap;
  const cudaError_t e = code_map(&wmap, w->codes, w->rows, w->K, kM);
  if (e != cudaSuccess) return e;
  GemmArgs a = dense_args(w, p, N, y, yd, ldy, ws, part);
  a.ats = x_scale;
  a.x = x;
  a.x_dtype = xd;
  a.ldx = ldx;
  a.K = w->K;
  return w->format == HQ_FP4_NV ? fused_launch<HQ_FP4_NV>(wmap, a, p.grid, st)
                                : fused_launch<HQ_FP4_MX>(wmap, a, p.grid, st);
}

// y = W a for a packed token matrix; part and counters as the plan needs them.
cudaError_t launch_matmul(const hq_fp4_matrix* w, const uint8_t* codes, const uint8_t* scales, const float* ats,
                          int N, void* y, hq_dtype yd, size_t ldy, uint8_t* ws, uint8_t* part, bool early,
                          cudaStream_t st) {
  const Plan p = plan_of(w->rows, N, w->K);
  CUtensorMap wmap, amap;
  cudaError_t e = code_map(&wmap, w->codes, w->rows, w->K, kM);
  if (e != cudaSuccess) return e;
  e = code_map(&amap, codes, N, w->K, p.pair ? p.nt_size / 2 : p.nt_size);
  if (e != cudaSuccess) return e;
  GemmArgs a = dense_args(w, p, N, y, yd, ldy, ws, part);
  a.asf = scales;
  a.ats = ats;
  a.early = early ? 1 : 0;
  if (p.pair) {
    return w->format == HQ_FP4_NV ? pair_launch<HQ_FP4_NV>(wmap, amap, a, p.grid, st)
                                  : pair_launch<HQ_FP4_MX>(wmap, amap, a, p.grid, st);
  }
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

// ------------------------------------------------------------------ experts

// Sizes of an expert layer: hidden H, intermediate I, and the rows that hold
// every routing (segments start at whole scale tiles).
struct Layer {
  int E, H, I, T, k, fmt;
  long rows;
};

// Workspace: [status, counters] [sort] [pos] [offsets, counts] [tokens' codes
// and scales by expert row] [h's codes and scales] [d, the experts' outputs].
// d is fp32 whatever y's type: it is a partial result of each token's sum.  In
// a 16-bit y's type (half the traffic of the two largest passes) bf16 results
// were 1.4 times as far off as one rounding of them, and an fp16 d beyond
// 65504 was infinite where the token's sum was not.
struct LayerWs {
  size_t sort, pos, ends, xc, xs, hc, hs, d, bytes;
};

LayerWs layer_ws(const Layer& l) {
  LayerWs w{};
  size_t at = kStatusBytes + kCounterBytes;
  auto take = [&](size_t n) {
    const size_t a = at;
    at += align256(n);
    return a;
  };
  const long pairs = static_cast<long>(l.T) * l.k;
  w.sort = take(route::sort_workspace_bytes(pairs, l.E));
  w.pos = take(pairs * 4);
  w.ends = take((2 * static_cast<size_t>(l.E) + 1) * 4);
  w.xc = take(static_cast<size_t>(l.rows) * (l.H / 2));
  w.xs = take(scale_bytes(l.fmt, l.rows, l.H));
  w.hc = take(static_cast<size_t>(l.rows) * (l.I / 2));
  w.hs = take(scale_bytes(l.fmt, l.rows, l.I));
  w.d = take(static_cast<size_t>(l.rows) * l.H * sizeof(float));
  w.bytes = at;
  return w;
}

hq_status check_layer(const hq_fp4_matrix* gate, const hq_fp4_matrix* up, const hq_fp4_matrix* down, int E, int T,
                      int k, Layer& l) {
  for (const hq_fp4_matrix* m : {gate, up, down}) {
    const hq_status ok = check_matrix(m);
    if (ok != HQ_OK) return ok;
  }
  if (E < 1 || T < 0 || k < 1) return HQ_ERR_INVALID_ARG;
  if (gate->format != up->format || gate->format != down->format || gate->rows != up->rows || gate->K != up->K ||
      gate->rows % E != 0 || down->rows % E != 0 || gate->rows / E != down->K || down->rows / E != gate->K) {
    return HQ_ERR_INVALID_ARG;
  }
  l = Layer{E, gate->K, down->K, T, k, gate->format, 0};
  if (l.H < 128 || l.I < 128) return HQ_ERR_UNSUPPORTED;
  if (E > kMaxGroups || k > 32 || l.H % 128 != 0 || l.I % 128 != 0 || T > (1 << 20)) return HQ_ERR_UNSUPPORTED;
  for (const hq_fp4_matrix* m : {gate, up, down}) {
    if (m->tensor_scale != nullptr && m->n_tensor_scales != 1 && m->n_tensor_scales != E) return HQ_ERR_INVALID_ARG;
  }
  const long pairs = static_cast<long>(T) * k;
  if (!route::sort_supported(pairs, E, kM)) return HQ_ERR_UNSUPPORTED;
  l.rows = (pairs + std::min<long>(E, pairs) * (kM - 1) + kM - 1) / kM * kM;
  return HQ_OK;
}

cudaError_t launch_experts(const hq_fp4_matrix* gate, const hq_fp4_matrix* up, const hq_fp4_matrix* down,
                           const Layer& l, const void* x, hq_dtype xd, size_t ldx, const int32_t* ids,
                           const float* topk_w, const float* x_scale, const float* h_scale, void* y, hq_dtype yd,
                           uint8_t* ws, cudaStream_t st) {
  const LayerWs o = layer_ws(l);
  int32_t* pos = reinterpret_cast<int32_t*>(ws + o.pos);
  int32_t* offsets = reinterpret_cast<int32_t*>(ws + o.ends);
  int32_t* counts = offsets + l.E + 1;
  const int rows = static_cast<int>(l.rows);
  cudaError_t e = route::launch_sort(ids, l.T * l.k, l.E, kM, pos, offsets, counts, ws + o.sort, st);
  if (e != cudaSuccess) return e;
  e = launch_quantize(l.fmt, xd, x, ldx, l.T, l.H, x_scale, ws + o.xc, ws + o.xs, nullptr, pos, l.k, rows, st);
  if (e != cudaSuccess) return e;
  // Token tiles: 256 experts x (2048, 512), top-8, 1024 / 2048 / 3000 / 4096
  // tokens (32 to 128 an expert) 120 / 155 / 195 / 248 us with 64, 131 / 160 /
  // 197 / 238 with 128; 60 experts x (4096, 1024), top-4, 500 / 1000 / 1400 /
  // 2000 tokens (33 to 133) 99 / 126 / 145 / 177 with 64, 109 / 125 / 147 / 171
  // with 128.
  const int nt = static_cast<long>(l.T) * l.k > 88l * l.E ? 128 : 64;
  const int box = nt == 128 ? Shape<HQ_FP4_NV, 128, kGated>::kBox : Shape<HQ_FP4_NV, 64, kGated>::kBox;
  const int grid = std::min(sm_count(), kMaxGrid);
  CUtensorMap wmap, wmap2, amap;
  GemmArgs a{};
  // Both products start behind a kernel that lets them start only after its own
  // wait: by then the sort is complete, and so is all that came before the call.
  a.early = 1;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.offsets = offsets;
  a.counts = counts;
  a.E = l.E;

  if ((e = code_map(&wmap, gate->codes, gate->rows, l.H, kM)) != cudaSuccess) return e;
  if ((e = code_map(&wmap2, up->codes, up->rows, l.H, kM)) != cudaSuccess) return e;
  if ((e = code_map(&amap, ws + o.xc, l.rows, l.H, box)) != cudaSuccess) return e;
  a.wsf = gate->scales;
  a.wts = gate->tensor_scale;
  a.n_wts = gate->n_tensor_scales;
  a.wsf2 = up->scales;
  a.wts2 = up->tensor_scale;
  a.n_wts2 = up->n_tensor_scales;
  a.asf = ws + o.xs;
  a.ats = x_scale;
  a.wkb = scale_tiles(l.fmt, l.H);
  a.M = l.I;
  a.mt = l.I / kM;
  a.C = (l.H + kChunk - 1) / kChunk;
  a.k_steps = l.H / 64;
  a.hts = h_scale;
  a.h_codes = ws + o.hc;
  a.h_scales = ws + o.hs;
  a.h_kb = scale_tiles(l.fmt, l.I);
  a.withhold = take_test_fault() ? 1 : 0;
  e = l.fmt == HQ_FP4_NV ? group_launch<HQ_FP4_NV, kGated>(nt, wmap, wmap2, amap, a, grid, st)
                         : group_launch<HQ_FP4_MX, kGated>(nt, wmap, wmap2, amap, a, grid, st);
  if (e != cudaSuccess) return e;

  if ((e = code_map(&wmap, down->codes, down->rows, l.I, kM)) != cudaSuccess) return e;
  if ((e = code_map(&amap, ws + o.hc, l.rows, l.I, box)) != cudaSuccess) return e;
  a.wsf = down->scales;
  a.wts = down->tensor_scale;
  a.n_wts = down->n_tensor_scales;
  a.asf = ws + o.hs;
  a.ats = h_scale;
  a.wkb = a.h_kb;
  a.M = l.H;
  a.mt = l.H / kM;
  a.C = (l.I + kChunk - 1) / kChunk;
  a.k_steps = l.I / 64;
  a.withhold = 0;
  a.y = ws + o.d;
  a.y_dtype = HQ_F32;
  a.ldy = l.H;
  e = l.fmt == HQ_FP4_NV ? group_launch<HQ_FP4_NV, kGrouped>(nt, wmap, wmap, amap, a, grid, st)
                         : group_launch<HQ_FP4_MX, kGrouped>(nt, wmap, wmap, amap, a, grid, st);
  if (e != cudaSuccess) return e;
  return route::launch_combine(HQ_F32, yd, ws + o.d, pos, topk_w, y, l.T, l.k, l.H, rows, st);
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
  if (fp4::fused_fits(w->format, batch, w->K)) {
    return from_cuda(fp4::launch_fused(w, x, x_dtype, ldx, batch, x_scale, y, y_dtype, ldy, ws, part, st));
  }
  const cudaError_t e = fp4::launch_quantize(w->format, x_dtype, x, ldx, batch, w->K, x_scale, codes, scales,
                                             nullptr, nullptr, 1, batch, st);
  if (e != cudaSuccess) return from_cuda(e);
  // The quantiser lets this kernel start only after its own wait, so all that
  // came before it on the stream, the weights' writers too, is complete: the
  // weights may be read at once.
  return from_cuda(fp4::launch_matmul(w, codes, scales, x_scale, batch, y, y_dtype, ldy, ws, part, true, st));
}

int hq_fp4_linear_launches(const hq_fp4_matrix* w, int batch) {
  if (fp4::check_matrix(w) != HQ_OK || batch < 1) return 0;
  return fp4::fused_fits(w->format, batch, w->K) ? 1 : 2;
}

size_t hq_fp4_experts_workspace_size(const hq_fp4_matrix* gate, const hq_fp4_matrix* up, const hq_fp4_matrix* down,
                                     int n_experts, int T, int k, hq_dtype y_dtype) {
  fp4::Layer l{};
  if (y_dtype < HQ_F16 || y_dtype > HQ_F32 || fp4::check_layer(gate, up, down, n_experts, T, k, l) != HQ_OK) return 0;
  return fp4::layer_ws(l).bytes;
}

hq_status hq_fp4_experts(const hq_fp4_matrix* gate, const hq_fp4_matrix* up, const hq_fp4_matrix* down,
                         int n_experts, const void* x, hq_dtype x_dtype, size_t ldx, int T, const int32_t* topk_ids,
                         const float* topk_w, int k, const float* x_scale, const float* h_scale, void* y,
                         hq_dtype y_dtype, void* workspace, size_t ws_bytes, hq_stream_t stream) {
  fp4::Layer l{};
  const hq_status ok = fp4::check_layer(gate, up, down, n_experts, T, k, l);
  if (ok != HQ_OK) return ok;
  if (y_dtype < HQ_F16 || y_dtype > HQ_F32) return HQ_ERR_INVALID_ARG;
  for (const float* s : {x_scale, h_scale}) {
    if (s != nullptr && (l.fmt != HQ_FP4_NV || (reinterpret_cast<uintptr_t>(s) & 3) != 0)) return HQ_ERR_INVALID_ARG;
  }
  if (T == 0) return HQ_OK;
  const hq_status rows_ok = fp4::check_rows(x, x_dtype, ldx, l.H);
  if (rows_ok != HQ_OK) return rows_ok;
  auto bad = [](const void* p, uintptr_t a) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
  if (bad(topk_ids, 4) || bad(topk_w, 4) || bad(y, 16)) return HQ_ERR_INVALID_ARG;
  if (fp4::bad_workspace(workspace, ws_bytes, fp4::layer_ws(l).bytes)) return HQ_ERR_WORKSPACE;
  return from_cuda(fp4::launch_experts(gate, up, down, l, x, x_dtype, ldx, topk_ids, topk_w, x_scale, h_scale, y,
                                       y_dtype, static_cast<uint8_t*>(workspace),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int hq_fp4_experts_launches(int T, int k) {
  if (T < 1 || k < 1 || k > 32) return 0;
  return 4 + route::sort_launches(static_cast<long>(T) * k);
}

}  // extern "C"
