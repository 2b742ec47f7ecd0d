// Cache quantiser: fp8 E4M3 with one fp32 scale per row, or fp4 E2M1 with one
// E4M3 scale per 16 channels.
//
// [P1] quantisation paragraphs: the attention cache uses fp8 ("partly
// token-wise fp8") and the indexer cache fp4; [P3] "storing the main KV in
// FP4": E2M1 values with one E4M3 scale per 16 channels.  Arithmetic (fixed
// here because the pages give no rounding rule):
//   fp8 row:  scale = fp32(amax / 448) (1 when amax == 0);
//             code = E4M3_rn_satfinite(fp32(x / scale)).
//   fp4 group of 16: s = E4M3_rn_satfinite(fp32(amax / 6));
//             code = E2M1_rn_satfinite(fp32(x / value(s))), 0 when value(s) == 0.
//   fp8 with bf16 rotary channels ([P1]: the RoPE dimensions stay in bf16):
//             the fp8 row rule over the first D - 64 channels (amax over
//             those only), then the last 64 channels as bf16 (nearest even);
//             a row is D - 64 code bytes followed by the 64 bf16 values.
// Divisions are IEEE round-to-nearest: by a row's (or group's) scale s they
// use Markstein's method (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): with
// y = RN(1/s), q0 = RN(x y), the remainder r = x - s q0 is exact in one FMA
// and RN(q0 + r y) = RN(x / s), which holds while nothing under- or
// overflows: the quotients here are at most 448 in magnitude, scales outside
// [2^-64, 2^64] take __fdiv_rn instead (so y is a normal number), and
// quotients small enough for r to underflow round to a zero code either way.
// The sign of a zero quotient is restored after the correction.  Conversions use the hardware
// cvt.rn.satfinite instructions.  One warp per row.
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_row.cuh"

namespace dsv4kv {

namespace {

constexpr int kRowsPerBlock = 8;

template <int PER, bool IN_FP32, int FMT>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
    quantize_kernel(const void* __restrict__ in, int64_t rows, uint8_t* __restrict__ codes, void* __restrict__ scales) {
  constexpr int D = 32 * PER;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kRowsPerBlock + (threadIdx.x >> 5);
  if (row >= rows) return;
  float x[PER];
  if (IN_FP32) {
    const float* src = static_cast<const float*>(in) + size_t(row) * D + PER * lane;
#pragma unroll
    for (int v = 0; v < PER / 4; ++v) {
      const float4 f = *reinterpret_cast<const float4*>(src + 4 * v);
      x[4 * v] = f.x;
      x[4 * v + 1] = f.y;
      x[4 * v + 2] = f.z;
      x[4 * v + 3] = f.w;
    }
  } else {
    const uint16_t* src = static_cast<const uint16_t*>(in) + size_t(row) * D + PER * lane;
#pragma unroll
    for (int v = 0; v < PER / 4; ++v) {
      const uint2 u = *reinterpret_cast<const uint2*>(src + 4 * v);
      x[4 * v] = bf16lo(u.x);
      x[4 * v + 1] = bf16hi(u.x);
      x[4 * v + 2] = bf16lo(u.y);
      x[4 * v + 3] = bf16hi(u.y);
    }
  }
  quantize_row<PER, FMT>(x, lane, size_t(row), codes, scales);
}

template <int PER>
dsv4kv_status launch_per(const void* in, int in_fp32, int64_t rows, int fmt, void* codes, void* scales,
                         cudaStream_t stream) {
  const dim3 grid(unsigned((rows + kRowsPerBlock - 1) / kRowsPerBlock));
  const dim3 block(32 * kRowsPerBlock);
  uint8_t* c = static_cast<uint8_t*>(codes);
  if (fmt == DSV4KV_FP8_E4M3_ROW) {
    if (in_fp32) quantize_kernel<PER, true, DSV4KV_FP8_E4M3_ROW><<<grid, block, 0, stream>>>(in, rows, c, scales);
    else quantize_kernel<PER, false, DSV4KV_FP8_E4M3_ROW><<<grid, block, 0, stream>>>(in, rows, c, scales);
  } else if (fmt == DSV4KV_FP8_E4M3_ROW_ROPE_BF16) {
    if (in_fp32)
      quantize_kernel<PER, true, DSV4KV_FP8_E4M3_ROW_ROPE_BF16><<<grid, block, 0, stream>>>(in, rows, c, scales);
    else
      quantize_kernel<PER, false, DSV4KV_FP8_E4M3_ROW_ROPE_BF16><<<grid, block, 0, stream>>>(in, rows, c, scales);
  } else {
    if (in_fp32) quantize_kernel<PER, true, DSV4KV_FP4_E2M1_G16><<<grid, block, 0, stream>>>(in, rows, c, scales);
    else quantize_kernel<PER, false, DSV4KV_FP4_E2M1_G16><<<grid, block, 0, stream>>>(in, rows, c, scales);
  }
  return check_launch("quantize_kernel");
}

}  // namespace

dsv4kv_status quantize_launch(const void* in, int in_fp32, int64_t rows, int dim, int fmt, void* codes,
                              void* scales, cudaStream_t stream) {
  if (rows == 0) return DSV4KV_OK;
  switch (dim) {
    case 128: return launch_per<4>(in, in_fp32, rows, fmt, codes, scales, stream);
    case 256: return launch_per<8>(in, in_fp32, rows, fmt, codes, scales, stream);
    case 512: return launch_per<16>(in, in_fp32, rows, fmt, codes, scales, stream);
    case 1024: return launch_per<32>(in, in_fp32, rows, fmt, codes, scales, stream);
    default: return set_error(DSV4KV_ERR_UNSUPPORTED, "quantize: dim must be 128, 256, 512 or 1024 (got %d)", dim);
  }
}

}  // namespace dsv4kv
