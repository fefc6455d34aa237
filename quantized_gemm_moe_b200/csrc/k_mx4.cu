// MXFP4 quantization of a matrix (weights or activations) and back.
#include <algorithm>

#include "qe_internal.h"
#include "qe_ptx.cuh"
#include "qe_quant.cuh"

namespace qe {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantIters = 4;                        // 256-channel pieces of a row per warp
constexpr int kQuantSpan = 256 * kQuantIters;         // channels per warp

// A warp takes 1024 neighbouring channels of a row: eight per lane and piece, so every load is 512
// contiguous bytes of bf16 (1 KB of fp32) and every store of codes 128. All loads are in flight before
// the first is used. HBM bound: 2 (4) bytes read and 0.53 written for each element.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) k_mx4_quantize(const void* __restrict__ X, const float* __restrict__ s,
                                                                int cols, int spans, size_t units,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const size_t unit = blockIdx.x * static_cast<size_t>(kQuantThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const size_t row = unit / spans;
  const int k0 = static_cast<int>(unit - row * spans) * kQuantSpan + lane * 8;
  const size_t base = row * cols, KT = (cols + kMxTileCols - 1) / kMxTileCols;
  uint4 raw[kQuantIters][BF16 ? 1 : 2];
#pragma unroll
  for (int j = 0; j < kQuantIters; ++j) {
    const int k = k0 + 256 * j;
    if (k < cols) {
      if constexpr (BF16) {
        raw[j][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + base + k));
      } else {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(X) + base + k);
        raw[j][0] = __ldg(q);
        raw[j][1] = __ldg(q + 1);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantIters; ++j) {
    const int k = k0 + 256 * j;
    float v[8];
    if (k < cols) {
      if constexpr (BF16) {
        const uint32_t w[4] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
          v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
        }
      } else {
        const uint4 p = raw[j][0], q = raw[j][1];
        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
      }
      if (s) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(s + k)), b = __ldg(reinterpret_cast<const float4*>(s + k) + 1);
        const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], f[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    uint32_t word;
    const uint32_t c = mx_quantize8(v, k < cols, lane, word);
    if (k < cols) {
      *reinterpret_cast<uint32_t*>(codes + (base + k) / 2) = c;
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(scales + mx_scale_word(row, k / kMxTileCols, KT)) = word;
    }
  }
}

// Two E2M1 codes (the low byte of c) as fp32.
__device__ __forceinline__ float2 e2m1x2(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}" : "=r"(h) : "r"(c));
  float2 f;
  asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// The values of the codes, eight channels per lane as above. Every value has two significant bits, so
// it is exact in bf16 and fp32 (2^-128, the smallest, is a subnormal of both).
__global__ void __launch_bounds__(kQuantThreads) k_mx4_dequantize(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int cols,
                                                                  int spans, size_t units, void* __restrict__ out,
                                                                  int out_bf16) {
  const int lane = threadIdx.x & 31;
  const size_t unit = blockIdx.x * static_cast<size_t>(kQuantThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const size_t row = unit / spans;
  const int k0 = static_cast<int>(unit - row * spans) * kQuantSpan + lane * 8;
  const size_t base = row * cols, KT = (cols + kMxTileCols - 1) / kMxTileCols;
  uint32_t c[kQuantIters], b[kQuantIters];
#pragma unroll
  for (int j = 0; j < kQuantIters; ++j) {
    const int k = k0 + 256 * j;
    if (k < cols) {
      c[j] = __ldg(reinterpret_cast<const uint32_t*>(codes + (base + k) / 2));
      b[j] = __ldg(scales + mx_scale_word(row, k / kMxTileCols, KT) + k % kMxTileCols / kMxBlock);
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantIters; ++j) {
    const int k = k0 + 256 * j;
    if (k >= cols) break;
    const float e = mx_scale(b[j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e2m1x2((c[j] >> (8 * i)) & 0xFFu);
      v[2 * i] = f.x * e;
      v[2 * i + 1] = f.y * e;
    }
    if (out_bf16) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
               (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + base + k) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + base + k);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* X, bool x_bf16, const float* s, int rows, int cols, uint8_t* codes,
                                uint8_t* scales, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int spans = static_cast<int>(ceil_div(cols, kQuantSpan));
  const size_t units = static_cast<size_t>(rows) * spans;
  const unsigned grid = static_cast<unsigned>(ceil_div(units, kQuantThreads / 32));
  if (x_bf16) k_mx4_quantize<true><<<grid, kQuantThreads, 0, st>>>(X, s, cols, spans, units, codes, scales);
  else k_mx4_quantize<false><<<grid, kQuantThreads, 0, st>>>(X, s, cols, spans, units, codes, scales);
  return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out,
                                  bool out_bf16, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int spans = static_cast<int>(ceil_div(cols, kQuantSpan));
  const size_t units = static_cast<size_t>(rows) * spans;
  k_mx4_dequantize<<<static_cast<unsigned>(ceil_div(units, kQuantThreads / 32)), kQuantThreads, 0, st>>>(
      codes, scales, cols, spans, units, out, out_bf16);
  return cudaGetLastError();
}

}  // namespace qe
