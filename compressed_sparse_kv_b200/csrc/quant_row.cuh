// One cache row quantised by one warp (shared by the bulk quantiser and the
// paged append).  The rounding rules and the division method are described in
// quantize.cu.
#pragma once

#include "common.cuh"

namespace dsv4kv {

__device__ __forceinline__ uint32_t cvt_e4m3x2(float hi, float lo) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;  // lo in bits 0..7, hi in bits 8..15
}
__device__ __forceinline__ uint32_t cvt_e2m1x2(float hi, float lo) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r & 0xffu;  // lo in bits 0..3, hi in bits 4..7
}
// x / s rounded to nearest for every x of a row or group that shares s.
struct RnDivider {
  float s, y;  // the divisor and RN(1 / s)
  bool fast;
  __device__ __forceinline__ float operator()(float x) const {
    if (!fast) return __fdiv_rn(x, s);
    const float q0 = x * y;
    const float r = fmaf(-q0, s, x);
    // The correction turns a quotient of -0 into +0; the sign of x / s is
    // the sign of q0 (s > 0), so it is put back.
    return copysignf(fmaf(r, y, q0), q0);
  }
};
__device__ __forceinline__ RnDivider rn_divider(float s) {
  RnDivider d;
  d.s = s;
  d.y = __frcp_rn(s);
  d.fast = s >= 0x1p-64f && s <= 0x1p64f;  // false for NaN
  return d;
}

__device__ __forceinline__ float e4m3_value(uint32_t c) {
  const float v = __uint_as_float((c & 0x7fu) << 20) * 0x1p120f;
  return (c & 0x80u) ? -v : v;
}

// Row x (PER channels per lane, channels [PER lane, PER lane + PER)) of D = 32 PER
// channels into row `row` of a cache in format FMT.  All 32 lanes call it.
template <int PER, int FMT>
__device__ __forceinline__ void quantize_row(const float (&x)[PER], int lane, size_t row, uint8_t* __restrict__ codes,
                                             void* __restrict__ scales) {
  constexpr int D = 32 * PER;
  if (FMT == DSV4KV_FP8_E4M3_ROW_ROPE_BF16) {
    // lanes [0, BL) hold the fp8 body, lanes [BL, 32) the 64 rotary channels
    constexpr int BL = 32 - 64 / PER;
    const bool body = lane < BL;
    float amax = 0.f;
    if (body) {
#pragma unroll
      for (int e = 0; e < PER; ++e) amax = fmaxf(amax, fabsf(x[e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    const RnDivider div = rn_divider(scale);
    uint8_t* row_dst = codes + size_t(row) * (D + 64);
    if (body) {
      uint32_t packed[PER / 4];
#pragma unroll
      for (int v = 0; v < PER / 4; ++v) {
        const uint32_t lo = cvt_e4m3x2(div(x[4 * v + 1]), div(x[4 * v]));
        const uint32_t hi = cvt_e4m3x2(div(x[4 * v + 3]), div(x[4 * v + 2]));
        packed[v] = lo | (hi << 16);
      }
#pragma unroll
      for (int v = 0; v < PER / 4; ++v) reinterpret_cast<uint32_t*>(row_dst + PER * lane)[v] = packed[v];
    } else {
      // bf16 of fp32 input rounds to nearest even; bf16 input is reproduced exactly
      uint32_t* dst = reinterpret_cast<uint32_t*>(row_dst + (D - 64) + 2 * PER * (lane - BL));
#pragma unroll
      for (int v = 0; v < PER / 2; ++v) dst[v] = pack_bf16x2(x[2 * v], x[2 * v + 1]);
    }
    if (lane == 0) static_cast<float*>(scales)[row] = scale;
  } else if (FMT == DSV4KV_FP8_E4M3_ROW) {
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    const RnDivider div = rn_divider(scale);
    uint32_t packed[PER / 4];
#pragma unroll
    for (int v = 0; v < PER / 4; ++v) {
      const uint32_t lo = cvt_e4m3x2(div(x[4 * v + 1]), div(x[4 * v]));
      const uint32_t hi = cvt_e4m3x2(div(x[4 * v + 3]), div(x[4 * v + 2]));
      packed[v] = lo | (hi << 16);
    }
    uint8_t* dst = codes + size_t(row) * D + PER * lane;
#pragma unroll
    for (int v = 0; v < PER / 4; ++v) reinterpret_cast<uint32_t*>(dst)[v] = packed[v];
    if (lane == 0) static_cast<float*>(scales)[row] = scale;
  } else {
    // groups of 16 channels: inside a lane (PER >= 16) or across 16/PER lanes
    constexpr int G = PER >= 16 ? 16 : PER;        // channels of a group held by this lane
    constexpr int NG = PER / G;                    // groups (or group parts) per lane
    constexpr int LANES_PER_GROUP = 16 / G;
    float s_val[NG];
    uint32_t s_code[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < G; ++e) amax = fmaxf(amax, fabsf(x[G * g + e]));
#pragma unroll
      for (int o = 1; o < LANES_PER_GROUP; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      s_code[g] = cvt_e4m3x2(0.f, __fdiv_rn(amax, 6.f)) & 0xffu;
      s_val[g] = e4m3_value(s_code[g]);
    }
    RnDivider divs[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) divs[g] = rn_divider(s_val[g] > 0.f ? s_val[g] : 1.f);
    uint8_t* dst = codes + size_t(row) * (D / 2) + (PER / 2) * lane;
    uint32_t packed[PER / 8 > 0 ? PER / 8 : 1];
#pragma unroll
    for (int v = 0; v < (PER + 7) / 8; ++v) packed[v] = 0;
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
      const float s = s_val[e / G];
      const RnDivider& div = divs[e / G];
      const uint32_t byte = s > 0.f ? cvt_e2m1x2(div(x[e + 1]), div(x[e])) : 0u;
      packed[e / 8] |= byte << (8 * ((e / 2) & 3));
    }
    if (PER >= 8) {
#pragma unroll
      for (int v = 0; v < PER / 8; ++v) reinterpret_cast<uint32_t*>(dst)[v] = packed[v];
    } else {
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) dst[e] = uint8_t(packed[0] >> (8 * e));
    }
    uint8_t* sdst = static_cast<uint8_t*>(scales) + size_t(row) * (D / 16);
    if (PER >= 16) {
#pragma unroll
      for (int g = 0; g < NG; ++g) sdst[NG * lane + g] = uint8_t(s_code[g]);
    } else if (lane % LANES_PER_GROUP == 0) {
      sdst[lane / LANES_PER_GROUP] = uint8_t(s_code[0]);
    }
  }
}

}  // namespace dsv4kv
