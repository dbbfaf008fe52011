// fp4_quant.cu -- rows of real values to microscaled 4-bit floating point:
// E2M1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and a sign) with one scale per block
// (16 values and an E4M3 scale, or 32 values and a power-of-two E8M0 scale).
//
// A thread takes 16 consecutive values of a row: 16-byte loads, the block's
// largest magnitude in registers (E8M0 blocks: one shuffle with the next
// thread), 8 bytes of codes out.  The scales of four neighbouring blocks meet
// in one word through shuffles, which is the 4-byte cell that the tensor
// cores' scale tile keeps together (include/hq.h).
//
// Bound: HBM.  Each value is read once and leaves as half a byte, a share of a
// scale and, if asked for, its rounded value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "fp4.cuh"
#include "fp4_quant.cuh"
#include "hq_common.cuh"
#include "hq_internal.h"
#include "hq_io.cuh"
#include "hq_launch.cuh"

namespace hq {
namespace fp4 {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16]) {
  constexpr int PER = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16 / PER; ++i) {
    uint4 u;
    T* t = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int j = 0; j < PER; ++j) t[j] = from_f32<T>(v[i * PER + j]);
    reinterpret_cast<uint4*>(p)[i] = u;
  }
}

struct QuantArgs {
  const void* x;
  size_t ldx;
  int rows;       // source rows
  int rows_pad;   // rows whose scales are written (whole tiles; beyond `rows`: zero)
  int K;
  int c_pad;      // 16-value chunks per row of whole scale tiles
  int cpb, rpb;   // chunks and rows of one block (a piece of one row, or whole rows)
  uint32_t inv;   // 65536 / cpb rounded up: tid / cpb for a block's threads
  const float* ts;
  uint8_t* codes;
  uint8_t* scales;
  int kb;          // scale tiles along K
  void* values;
  const int32_t* pos;  // destination rows [rows][k], or nullptr: row r to row r
  int k;
  int dst_rows;
};


// Where a row's codes go: to its own row; there with the rounded values; or to
// the rows of the token's pairs.
enum Target { kRows = 0, kValues = 1, kScatter = 2 };

template <typename T, int FMT, int TARGET>
__device__ __forceinline__ void quantize_piece(const QuantArgs& a, long row, int c, bool mine, const SixTs& ts,
                                               const Raw16<T>& raw) {
  const bool live = mine && row < a.rows && c * 16 < a.K;
  float v[16];
  raw.unpack(v);
  const Packed16 p = pack16<FMT>(v, raw.top(), ts, 1);
  const uint32_t byte = live ? p.byte : 0u;
  // four blocks' scales in one word
  constexpr int S = FMT == HQ_FP4_NV ? 0 : 1;  // log2 of the threads per block
  uint32_t sw = byte << (8 * (c >> S & 3));
  sw |= __shfl_xor_sync(~0u, sw, 1 << S);
  sw |= __shfl_xor_sync(~0u, sw, 2 << S);
  const bool scale_lane = mine && (c & ((4 << S) - 1)) == 0;
  const int st = c >> (2 + S);  // scale tile along K
  if constexpr (TARGET != kScatter) {
    const long o = row * a.K + c * 16;
    if (live) *reinterpret_cast<uint2*>(a.codes + (o >> 1)) = p.codes;
    if (scale_lane && row < a.rows_pad) *reinterpret_cast<uint32_t*>(a.scales + scale_cell(row, st, a.kb)) = sw;
    if (TARGET == kValues && live) {
      const uint64_t e2 = f2(p.eff, p.eff);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = from_e2m1x2((i < 4 ? p.codes.x : p.codes.y) >> (8 * (i & 3)));
        un2(mul2(f2(f.x, f.y), e2), v[2 * i], v[2 * i + 1]);
      }
      store16<T>(static_cast<T*>(a.values) + o, v);
    }
  } else if (row < a.rows) {
    for (int j = 0; j < a.k; ++j) {
      const int dst = __ldg(a.pos + row * a.k + j);
      if (static_cast<uint32_t>(dst) >= static_cast<uint32_t>(a.dst_rows)) continue;
      if (live) *reinterpret_cast<uint2*>(a.codes + static_cast<long>(dst) * (a.K / 2) + c * 8) = p.codes;
      if (scale_lane) *reinterpret_cast<uint32_t*>(a.scales + scale_cell(dst, st, a.kb)) = sw;
    }
  }
}

template <typename T, int FMT, int TARGET>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const QuantArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  // Rows from the last to the first: what wrote x, or read it for its largest
  // value, did the end last, and that part may still lie in L2.
  const int r = static_cast<int>(threadIdx.x * a.inv >> 16);
  const int c = blockIdx.y * a.cpb + threadIdx.x - r * a.cpb;
  const long row = static_cast<long>(gridDim.x - 1 - blockIdx.x) * a.rpb + r;
  const bool mine = r < a.rpb && c < a.c_pad;
  Raw16<T> v;
  if (mine && row < a.rows && c * 16 < a.K) {
    v.load(static_cast<const T*>(a.x) + row * a.ldx + c * 16);
  } else {
    v.zero();
  }
  const SixTs ts(FMT == HQ_FP4_NV ? a.ts : nullptr);
  quantize_piece<T, FMT, TARGET>(a, row, c, mine, ts, v);
}

// The largest magnitude of a tensor over 2688 (= 6 * 448, the largest value
// of a code times the largest block scale), 1 for an all-zero tensor.  Every
// block folds its maximum into ws[0] (magnitudes order as their bit patterns;
// a NaN's is above all), the last one writes the result.  Both words of ws are
// zero at the start.
template <typename T>
__global__ void __launch_bounds__(kThreads) tensor_scale_kernel(const T* __restrict__ x, size_t ldx, int rows,
                                                                int chunks, float* __restrict__ out,
                                                                uint32_t* __restrict__ ws) {
  pdl_wait();
  pdl_launch_dependents();
  const size_t total = static_cast<size_t>(rows) * chunks;
  uint32_t m = 0;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * kThreads) {
    const size_t r = i / chunks;
    float v[16];
    load_chunk<T, 16>(x + r * ldx + (i - r * chunks) * 16, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
  m = __reduce_max_sync(~0u, m);
  __shared__ uint32_t part[kThreads / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) m = max(m, part[i]);
    atomicMax(ws, m);
    __threadfence();
    if (atomicAdd(ws + 1, 1u) == gridDim.x - 1) {
      __threadfence();
      const float s = __fdiv_rn(__uint_as_float(atomicMax(ws, 0u)), 2688.f);
      *out = s == 0.f ? 1.f : s;
    }
  }
}

template <typename T, int FMT>
cudaError_t quantize_launch(const QuantArgs& a, dim3 grid, cudaStream_t st) {
  const dim3 block((a.cpb * a.rpb + 31) / 32 * 32);
  if (a.pos != nullptr) return launch_pdl(quantize_rows_kernel<T, FMT, kScatter>, grid, block, 0, st, true, a);
  return a.values != nullptr ? launch_pdl(quantize_rows_kernel<T, FMT, kValues>, grid, block, 0, st, true, a)
                             : launch_pdl(quantize_rows_kernel<T, FMT, kRows>, grid, block, 0, st, true, a);
}

template <typename T>
cudaError_t quantize_launch(int fmt, const QuantArgs& a, dim3 grid, cudaStream_t st) {
  return fmt == HQ_FP4_NV ? quantize_launch<T, HQ_FP4_NV>(a, grid, st) : quantize_launch<T, HQ_FP4_MX>(a, grid, st);
}

}  // namespace

cudaError_t launch_quantize(int fmt, hq_dtype xd, const void* x, size_t ldx, int rows, int K, const float* ts,
                            uint8_t* codes, uint8_t* scales, void* values, const int32_t* pos, int k,
                            int dst_rows, cudaStream_t st) {
  QuantArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.rows_pad = pos == nullptr ? (rows + 127) / 128 * 128 : rows;
  a.K = K;
  a.kb = scale_tiles(fmt, K);
  a.c_pad = a.kb * (fmt == HQ_FP4_NV ? 4 : 8);
  const int pieces = (a.c_pad + kThreads - 1) / kThreads;
  a.cpb = ((a.c_pad + pieces - 1) / pieces + 7) / 8 * 8;  // whole scale words
  a.rpb = pieces > 1 ? 1 : std::max(1, kThreads / a.cpb);
  a.inv = (65536 + a.cpb - 1) / a.cpb;
  a.ts = ts;
  a.codes = codes;
  a.scales = scales;
  a.values = values;
  a.pos = pos;
  a.k = k;
  a.dst_rows = dst_rows;
  const dim3 grid((a.rows_pad + a.rpb - 1) / a.rpb, pieces);
  switch (xd) {
    case HQ_F16: return quantize_launch<__half>(fmt, a, grid, st);
    case HQ_BF16: return quantize_launch<__nv_bfloat16>(fmt, a, grid, st);
    default: return quantize_launch<float>(fmt, a, grid, st);
  }
}

hq_status check_rows(const void* x, hq_dtype xd, size_t ldx, int K) {
  if (xd < HQ_F16 || xd > HQ_F32) return HQ_ERR_INVALID_ARG;
  const size_t es = xd == HQ_F32 ? 4 : 2;
  if (x == nullptr || (reinterpret_cast<uintptr_t>(x) & 15) != 0) return HQ_ERR_INVALID_ARG;
  if (ldx < static_cast<size_t>(K) || (ldx * es) % 16 != 0 || ldx > (size_t{1} << 40)) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

hq_status check_shape(int fmt, long rows, int K) {
  if (fmt != HQ_FP4_NV && fmt != HQ_FP4_MX) return HQ_ERR_INVALID_ARG;
  if (rows < 0 || rows > (1 << 28) || K <= 0) return HQ_ERR_INVALID_ARG;
  if (K % 32 != 0 || K > (1 << 17)) return HQ_ERR_UNSUPPORTED;
  return HQ_OK;
}

hq_status check_matrix(const hq_fp4_matrix* m) {
  if (m == nullptr) return HQ_ERR_INVALID_ARG;
  const hq_status s = check_shape(m->format, m->rows, m->K);
  if (s != HQ_OK) return s;
  if (m->rows > 0 && (m->codes == nullptr || m->scales == nullptr)) return HQ_ERR_INVALID_ARG;
  auto bad = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
  if (bad(m->codes, 16) || bad(m->scales, 16) || bad(m->tensor_scale, 4)) return HQ_ERR_INVALID_ARG;
  if (m->tensor_scale != nullptr && (m->format != HQ_FP4_NV || m->n_tensor_scales < 1)) return HQ_ERR_INVALID_ARG;
  return HQ_OK;
}

}  // namespace fp4
}  // namespace hq

using namespace hq;

extern "C" {

size_t hq_fp4_scale_bytes(int format, int rows, int K) {
  if (fp4::check_shape(format, rows, K) != HQ_OK) return 0;
  return fp4::scale_bytes(format, rows, K);
}

hq_status hq_fp4_quantize(const void* x, hq_dtype x_dtype, size_t ldx, const hq_fp4_matrix* q, void* values,
                          hq_stream_t stream) {
  const hq_status ok = fp4::check_matrix(q);
  if (ok != HQ_OK) return ok;
  if (q->tensor_scale != nullptr && q->n_tensor_scales != 1) return HQ_ERR_UNSUPPORTED;
  if (q->rows == 0) return HQ_OK;
  const hq_status rows_ok = fp4::check_rows(x, x_dtype, ldx, q->K);
  if (rows_ok != HQ_OK) return rows_ok;
  if (values != nullptr && (reinterpret_cast<uintptr_t>(values) & 15) != 0) return HQ_ERR_INVALID_ARG;
  return from_cuda(fp4::launch_quantize(q->format, x_dtype, x, ldx, q->rows, q->K, q->tensor_scale, q->codes,
                                        q->scales, values, nullptr, 1, q->rows,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

hq_status hq_fp4_tensor_scale(const void* x, hq_dtype x_dtype, size_t ldx, int rows, int K, float* scale,
                              void* workspace, size_t ws_bytes, hq_stream_t stream) {
  const hq_status ok = fp4::check_shape(HQ_FP4_NV, rows, K);
  if (ok != HQ_OK) return ok;
  if (rows == 0) return HQ_ERR_INVALID_ARG;
  const hq_status rows_ok = fp4::check_rows(x, x_dtype, ldx, K);
  if (rows_ok != HQ_OK) return rows_ok;
  if (scale == nullptr || (reinterpret_cast<uintptr_t>(scale) & 3) != 0) return HQ_ERR_INVALID_ARG;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || ws_bytes < 256) {
    return HQ_ERR_WORKSPACE;
  }
  const int chunks = K / 16;
  const size_t blocks = (static_cast<size_t>(rows) * chunks + fp4::kThreads - 1) / fp4::kThreads;
  const int grid = static_cast<int>(std::min<size_t>(blocks, static_cast<size_t>(sm_count()) * 8));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint32_t* ws = static_cast<uint32_t*>(workspace);
  if (const cudaError_t e = cudaMemsetAsync(ws, 0, 2 * sizeof(uint32_t), st); e != cudaSuccess) return from_cuda(e);
  auto go = [&](auto* p) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    return launch_pdl(fp4::tensor_scale_kernel<T>, dim3(grid), dim3(fp4::kThreads), 0, st, true, p, ldx, rows,
                      chunks, scale, ws);
  };
  switch (x_dtype) {
    case HQ_F16: return from_cuda(go(static_cast<const __half*>(x)));
    case HQ_BF16: return from_cuda(go(static_cast<const __nv_bfloat16*>(x)));
    default: return from_cuda(go(static_cast<const float*>(x)));
  }
}

}  // extern "C"
