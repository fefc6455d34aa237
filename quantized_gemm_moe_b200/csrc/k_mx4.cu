// MXFP4 quantization of a matrix (weights or activations) and back.
#include <algorithm>

#include "qe_internal.h"
#include "qe_launch.cuh"
#include "qe_ptx.cuh"
#include "qe_quant.cuh"

namespace qe {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kLaneK = 8;                             // channels per lane and step: a quarter of a block
constexpr int kStepK = 32 * kLaneK;                   // channels per warp and step
constexpr int kQuantSteps = 2;
constexpr int kQuantRows = 2;                         // neighbouring rows per warp: they share the factors s
constexpr int kQuantSpan = kStepK * kQuantSteps;      // channels per warp

// A warp takes 512 neighbouring channels of two rows: eight per lane and step, four lanes to a block, so that a
// step reads 512 contiguous bytes of bf16 (1 KB of fp32) and writes 128 of codes. All loads of x are in flight
// before the first is used. HBM: 2 (4) bytes read and 0.53 written for each element; what comes next is L1,
// which the factors s (1 KB a step) load more than bf16 rows do, hence two rows. 29568 x 8192 bf16 with s:
// 96 us, 6.4 TB/s with the registers bounded for five CTAs on an SM. (Read through the non-coherent path, which memory
// that the kernel before may still be writing does not allow, it took 94; there four and six CTAs took 101, and one row
// and 1024 channels 111.) The bound, 48 registers, is measured on bf16; with it the fp32 form with factors keeps 104 bytes a
// thread in local memory: 8192 x 8192 52 us, 44 without factors.
// FULL: the warp's channels and rows all exist (nothing is predicated).
template <bool BF16, bool SMOOTH, bool FULL>
__device__ __forceinline__ void quantize_span(const uint8_t* x, size_t pitch, const float* s,
                                              int k0, int cols, int rows, int lane, uint8_t* __restrict__ c,
                                              uint8_t* __restrict__ sc0, uint8_t* __restrict__ sc1) {
  constexpr int kE = BF16 ? 2 : 4;
  uint4 raw[kQuantSteps][kQuantRows][kE / 2];
#pragma unroll
  for (int j = 0; j < kQuantSteps; ++j) {
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
      if (FULL || (k0 + kStepK * j < cols && r < rows)) {
#pragma unroll
        for (int h = 0; h < kE / 2; ++h)
          raw[j][r][h] = *(reinterpret_cast<const uint4*>(x + r * pitch * kE + kStepK * kE * j) + h);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kQuantSteps; ++j) {
    const int k = k0 + kStepK * j;
    float f[8];
    if (SMOOTH && (FULL || k < cols)) {
      const float4 f0 = *reinterpret_cast<const float4*>(s + kStepK * j);
      const float4 f1 = *(reinterpret_cast<const float4*>(s + kStepK * j) + 1);
      f[0] = f0.x; f[1] = f0.y; f[2] = f0.z; f[3] = f0.w;
      f[4] = f1.x; f[5] = f1.y; f[6] = f1.z; f[7] = f1.w;
    }
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
      const bool valid = FULL || (k < cols && r < rows);
      float v[8];
      if (valid) {
        const uint4 p = raw[j][r][0], q = raw[j][r][kE / 2 - 1];
        if constexpr (BF16) {
          const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        } else {
          const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        }
        if constexpr (SMOOTH) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], f[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      }
      uint32_t top = absmax8(v);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t byte = mx_scale_byte(top);
      const uint32_t code = mx_codes8(v, byte);
      if (valid) *reinterpret_cast<uint32_t*>(c + r * pitch / 2 + kStepK / 2 * j) = code;
      if ((lane & 3) == 0 && (FULL || (k < static_cast<int>(round_up(cols, kMxTileCols)) && r < rows)))
        (r ? sc1 : sc0)[kStepK / kMxTileCols * kMxTileBytes * j] = static_cast<uint8_t>(valid ? byte : kMxOne);
    }
  }
}

template <bool BF16, bool SMOOTH>
__global__ void __launch_bounds__(kQuantThreads, 5) k_mx4_quantize(const void* X, const float* s,
                                                                int rows, int cols, uint32_t spans, uint32_t units,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();  // a product may set itself up, and load its weights, meanwhile
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const uint32_t pair = unit / spans;  // in 32 bits: a 64-bit division costs as much as a step's arithmetic
  const size_t row = static_cast<size_t>(pair) * kQuantRows;
  const int span0 = static_cast<int>(unit - pair * spans) * kQuantSpan, k0 = span0 + lane * kLaneK;
  const size_t at = row * cols + k0;
  const uint8_t* x = static_cast<const uint8_t*>(X) + at * (BF16 ? 2 : 4);
  const int KT = (cols + kMxTileCols - 1) / kMxTileCols, left = static_cast<int>(rows - row);
  uint8_t* sc0 = scales + mx_scale_row(row, KT) + mx_scale_at(k0);
  uint8_t* sc1 = scales + mx_scale_row(row + 1, KT) + mx_scale_at(k0);
  if (span0 + kQuantSpan <= cols && left >= kQuantRows)
    quantize_span<BF16, SMOOTH, true>(x, cols, s + k0, k0, cols, left, lane, codes + at / 2, sc0, sc1);
  else
    quantize_span<BF16, SMOOTH, false>(x, cols, s + k0, k0, cols, left, lane, codes + at / 2, sc0, sc1);
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

// The values of the codes, eight channels per lane and step. Every value has two significant bits, so
// it is exact in bf16 and fp32 (2^-128, the smallest, is a subnormal of both).
constexpr int kDequantSpan = 1024;  // channels per warp
__global__ void __launch_bounds__(kQuantThreads) k_mx4_dequantize(const uint8_t* codes,
                                                                  const uint8_t* scales, int cols,
                                                                  uint32_t spans, uint32_t units, void* __restrict__ out,
                                                                  int out_bf16) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const uint32_t row32 = unit / spans;
  const size_t row = row32;
  constexpr int kSteps = kDequantSpan / 256;
  const int k0 = static_cast<int>(unit - row32 * spans) * kDequantSpan + lane * 8;
  const size_t base = row * cols;
  const uint8_t* sc = scales + mx_scale_row(row, (cols + kMxTileCols - 1) / kMxTileCols);
  uint32_t c[kSteps], b[kSteps];
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
    const int k = k0 + 256 * j;
    if (k < cols) {
      c[j] = *reinterpret_cast<const uint32_t*>(codes + (base + k) / 2);
      b[j] = sc[mx_scale_at(k)];
    }
  }
#pragma unroll
  for (int j = 0; j < kSteps; ++j) {
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
      for (int i = 0; i < 4; ++i) w[i] = bf16x2_word(v[2 * i], v[2 * i + 1]);
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
  const size_t units = static_cast<size_t>(ceil_div(rows, kQuantRows)) * spans;
  if (units > 0xFFFF0000u) return cudaErrorInvalidValue;  // four terabytes of bf16
  const unsigned grid = static_cast<unsigned>(ceil_div(units, kQuantThreads / 32));
  auto k = x_bf16 ? (s ? k_mx4_quantize<true, true> : k_mx4_quantize<true, false>)
                  : (s ? k_mx4_quantize<false, true> : k_mx4_quantize<false, false>);
  return launch_dependent(k, dim3(grid), kQuantThreads, 0, 1, st, X, s, rows, cols, static_cast<uint32_t>(spans), static_cast<uint32_t>(units),
                          codes, scales);
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out,
                                  bool out_bf16, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int spans = static_cast<int>(ceil_div(cols, kDequantSpan));
  const size_t units = static_cast<size_t>(rows) * spans;
  if (units > 0xFFFF0000u) return cudaErrorInvalidValue;
  return launch_dependent(k_mx4_dequantize, dim3(static_cast<unsigned>(ceil_div(units, kQuantThreads / 32))), kQuantThreads, 0,
                          1, st, codes, scales, cols, static_cast<uint32_t>(spans), static_cast<uint32_t>(units), out,
                          static_cast<int>(out_bf16));
}

}  // namespace qe
