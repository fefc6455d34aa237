// The residual's addition and the root-mean-square norm in front of a quantized projection, with the
// normed row quantized in the same pass, and the dequantization of per-token int8 codes.
#include <algorithm>

#include "qe_internal.h"
#include "qe_launch.cuh"
#include "qe_ptx.cuh"
#include "qe_quant.cuh"

namespace qe {
namespace {

struct NormArgs {
  const void* X;
  const void* R;       // residual, or nullptr
  const void* gamma;
  const float* s_inv;  // or nullptr
  double eps;
  int T, d, qmax, g_bf16;
  void* H;             // x + r in x's type, or nullptr
  void* Y;             // normed row in x's type, or nullptr
  uint8_t* codes;
  void* scales;        // sa fp32 [T] (int8 codes) or MXFP4 scale tiles
};

enum { kOutNone = 0, kOutInt8 = 1, kOutMx4 = 2 };

// Eight elements at p + i (16-byte aligned) in fp32.
__device__ __forceinline__ void ld8(const void* p, size_t i, bool bf16, float (&v)[8]) {
  if (bf16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
      v[2 * j + 1] = bf16_bits_to_f32(w[j] >> 16);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
__device__ __forceinline__ void st8(void* p, size_t i, bool bf16, const float (&v)[8]) {
  if (bf16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bf16x2_word(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Eight elements as loaded: their use is far from their load.
template <bool BF16>
struct Raw8 {
  uint4 v[BF16 ? 1 : 2];
};
template <bool BF16>
__device__ __forceinline__ void ld_raw(const void* p, size_t i, Raw8<BF16>& r) {
  if constexpr (BF16) {
    r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  } else {
    r.v[0] = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)[0];
    r.v[1] = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)[1];
  }
}
template <bool BF16>
__device__ __forceinline__ void unpack(const Raw8<BF16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const uint32_t u[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(w[i]);
      v[4 + i] = __uint_as_float(u[i]);
    }
  }
}
// v[i] = fl32(x[i] + v[i])
template <bool BF16>
__device__ __forceinline__ void add_raw(const Raw8<BF16>& x, float (&v)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {x.v[0].x, x.v[0].y, x.v[0].z, x.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)  // the bf16 operand is widened in the addition itself
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
          : "+f"(v[2 * i]), "+f"(v[2 * i + 1])
          : "r"(w[i]));
  } else {
    float f[8];
    unpack<false>(x, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(f[i], v[i]);
  }
}

// The row statistic from the warps' sums of squares (one warp): held in 64 bits and rounded once.
__device__ __forceinline__ void norm_rstd(const double* sum_s, int nw, int lane, const NormArgs& a, float* rstd) {
  double sum = lane < nw ? sum_s[lane] : 0.0;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) *rstd = static_cast<float>(rsqrt(sum / a.d + a.eps));
}

// A thread holds VPT vectors of eight neighbouring channels of a row, blockDim.x vectors apart, in registers
// from the row's only read to its last write.
//   h = fl32(x + r); rstd = fl32(1/sqrt(sum h^2 / d + eps)); y = fl32(fl32(h*rstd)*g); v = fl32(y*s_inv)
// The sum of squares is held in 64 bits and rstd rounded once, after which every value that decides a
// code is one fp32 operation, so the codes do not depend on the order of the sum.
// HBM bound: 8192 x 8192 bf16 with residual, A6: 99 us, 6.1 TB/s; MXFP4: 95 us, 6.0 TB/s. Persistent CTAs that load
// a row ahead, and several rows to a CTA, were slower (117-136 and 125 us for A6): the registers they take cost
// more resident warps than they save waits.
template <bool BF16, int VPT, int OUT>
__global__ void __launch_bounds__(1024) k_add_rmsnorm(const NormArgs a) {
  __shared__ double sum_s[32];
  __shared__ uint32_t top_s[32];
  __shared__ float rstd_s;
  grid_dep_wait();
  grid_dep_launch();  // the projection may set itself up meanwhile
  const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int KT = (a.d + kMxTileCols - 1) / kMxTileCols;
  Raw8<BF16> x[VPT], q[VPT];
  float h[VPT][8];
  auto load = [&](size_t row) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int k = (tid + j * nt) * 8;
      if (k < a.d) {
        ld_raw<BF16>(a.X, row * a.d + k, x[j]);
        if (a.R) ld_raw<BF16>(a.R, row * a.d + k, q[j]);
      }
    }
  };
  // h of a row, its copy to H, and this warp's sum of squares
  auto add = [&](size_t row) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int k = (tid + j * nt) * 8;
      if (k < a.d) {
        if (a.R) {
          unpack<BF16>(q[j], h[j]);
          add_raw<BF16>(x[j], h[j]);
          if (a.H) st8(a.H, row * a.d + k, BF16, h[j]);
        } else {
          unpack<BF16>(x[j], h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(h[j][i]), static_cast<double>(h[j][i]), sum);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) sum_s[warp] = sum;
  };
  // y and v of a row, and this warp's largest |v|: magnitudes order as unsigned bit patterns, with infinities
  // and NaNs above every finite value
  auto scale = [&](size_t row) {
    const float rstd = rstd_s;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int k = (tid + j * nt) * 8;
      if (k < a.d) {
        float g[8];
        ld8(a.gamma, k, a.g_bf16, g);
        mul8(h[j], rstd);
        mul8(h[j], g);
        if (a.Y) st8(a.Y, row * a.d + k, BF16, h[j]);
        if (OUT != kOutNone && a.s_inv) {
          ld8(a.s_inv, k, false, g);
          mul8(h[j], g);
        }
        if (OUT == kOutInt8) top = max(top, absmax8(h[j]));
      }
    }
    if (OUT == kOutInt8) {
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0) top_s[warp] = top;
    }
    if (OUT == kOutMx4) {
      // four neighbouring lanes hold a block (rows are whole blocks); the first writes its scale
      uint8_t* sc = static_cast<uint8_t*>(a.scales) + mx_scale_row(row, KT);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int k = (tid + j * nt) * 8;
        uint32_t t = k < a.d ? absmax8(h[j]) : 0u;
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        const uint32_t byte = mx_scale_byte(t);
        if (k < a.d) *reinterpret_cast<uint32_t*>(a.codes + (row * a.d + k) / 2) = mx_codes8(h[j], byte);
        if ((lane & 3) == 0 && k < KT * kMxTileCols) sc[mx_scale_at(k)] = static_cast<uint8_t>(k < a.d ? byte : kMxOne);
      }
    }
  };
  // the int8 codes of a row, with the scale of the layer's own quantization: the two give the same codes
  auto codes = [&](size_t row) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, lane < nw ? top_s[lane] : 0u);
    const bool finite = top < 0x7F800000u;
    const float sa = finite ? __fdiv_rn(__uint_as_float(top), static_cast<float>(a.qmax)) : __uint_as_float(0x7FC00000u);
    if (tid == 0) static_cast<float*>(a.scales)[row] = sa;
    const float inv = sa > 0.0f ? __frcp_rn(sa) : 0.0f;
    const float limit = rtn_fast_ok(sa, inv) ? rtn_limit(a.qmax) : 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int k = (tid + j * nt) * 8;
      if (k < a.d) {
        uint32_t w0 = 0, w1 = 0;
        if (finite) rtn_code8_row(h[j], sa, inv, limit, a.qmax, w0, w1);
        *reinterpret_cast<uint2*>(a.codes + row * a.d + k) = make_uint2(w0, w1);
      }
    }
  };

  const size_t row = blockIdx.x;
  load(row);
  add(row);
  __syncthreads();
  if (warp == 0) norm_rstd(sum_s, nw, lane, a, &rstd_s);
  __syncthreads();
  scale(row);
  if (OUT == kOutInt8) {
    __syncthreads();
    codes(row);
  }
}

// out[t][k] = codes[t][k] * sa[t], eight channels per thread and step, four steps in flight.
constexpr int kDequantSteps = 4;
__global__ void __launch_bounds__(256) k_act_dequant(const int8_t* codes, const float* sa,
                                                     uint32_t d8, uint32_t n8, void* __restrict__ out, int out_bf16) {
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t i0 = blockIdx.x * (256u * kDequantSteps) + threadIdx.x;
  uint2 w[kDequantSteps];
  float s[kDequantSteps];
#pragma unroll
  for (int j = 0; j < kDequantSteps; ++j) {
    const uint32_t i = i0 + 256u * j;
    if (i < n8) {
      w[j] = *(reinterpret_cast<const uint2*>(codes) + i);
      s[j] = sa[i / d8];
    }
  }
#pragma unroll
  for (int j = 0; j < kDequantSteps; ++j) {
    const uint32_t i = i0 + 256u * j;
    if (i >= n8) break;
    float v[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      v[b] = static_cast<float>(static_cast<int8_t>(w[j].x >> (8 * b))) * s[j];
      v[4 + b] = static_cast<float>(static_cast<int8_t>(w[j].y >> (8 * b))) * s[j];
    }
    st8(out, static_cast<size_t>(i) * 8, out_bf16, v);
  }
}

template <bool BF16, int VPT>
cudaError_t launch_norm_t(const NormArgs& a, int out, cudaStream_t st) {
  const int threads = static_cast<int>(round_up(ceil_div(a.d / 8, VPT), 32));
  auto k = out == kOutInt8 ? k_add_rmsnorm<BF16, VPT, kOutInt8>
           : out == kOutMx4 ? k_add_rmsnorm<BF16, VPT, kOutMx4>
                            : k_add_rmsnorm<BF16, VPT, kOutNone>;
  return launch_dependent(k, dim3(static_cast<unsigned>(a.T)), threads, 0, 1, st, a);
}

// Vectors per thread. With at most two rows per SM latency counts, and a row takes as many threads as it has
// vectors, up to 1024 (300 x 4096 int8: 5.4 us against 6.0 with two). With more rows, fewer and fatter warps pay
// less for the block reductions and keep as many bytes in flight (8192 x 8192 bf16 A6: 201 us with one vector,
// 127 with two, 104 with four, 118 with eight at half the warps; 4096 x 4096: 38, 31, 32); fp32 rows have twice
// the bytes for the same work and take two up to 8192 channels (4096 x 8192: 98 us, and 110 with four). Longer ones take four,
// for which 64 registers are too few in fp32 (68 to 104 bytes a thread in local memory): 300 x 8960 9.6 us, 4096 x 12288 162.
// bf16 rows near the longest leave one CTA on an SM, and its waits show: 2000 x 29568 119 us, 5.0 TB/s.
template <bool BF16>
cudaError_t launch_norm_x(const NormArgs& a, int out, cudaStream_t st) {
  const int vecs = a.d / 8;
  const bool few = a.T <= 2 * decode_grid_sms();
  if (vecs <= (few ? 1024 : 256)) return launch_norm_t<BF16, 1>(a, out, st);
  if (vecs <= (few ? 2048 : BF16 ? 512 : 1024)) return launch_norm_t<BF16, 2>(a, out, st);
  return launch_norm_t<BF16, 4>(a, out, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const void* X, bool x_bf16, const void* R, const void* gamma, bool g_bf16, double eps,
                               int T, int d, const float* s_inv, int a_bits, void* H, void* Y, void* codes,
                               void* scales, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  NormArgs a{};
  a.X = X;
  a.R = R;
  a.gamma = gamma;
  a.s_inv = s_inv;
  a.eps = eps;
  a.T = T;
  a.d = d;
  a.qmax = (1 << (a_bits - 1)) - 1;
  a.g_bf16 = g_bf16;
  a.H = H;
  a.Y = Y;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  const int out = a_bits == 16 ? kOutNone : a_bits == 4 ? kOutMx4 : kOutInt8;
  return x_bf16 ? launch_norm_x<true>(a, out, st) : launch_norm_x<false>(a, out, st);
}

cudaError_t launch_act_dequant(const int8_t* codes, const float* sa, int T, int d, void* out, bool out_bf16,
                               cudaStream_t st) {
  // the kernel counts vectors of eight in 32 bits: larger matrices go in ranges of rows
  const uint32_t d8 = static_cast<uint32_t>(d / 8);
  const int most = static_cast<int>(std::min<uint32_t>(0xFFFF0000u / d8, 1u << 30));
  for (int row = 0; row < T; row += std::min(most, T - row)) {
    const uint32_t n8 = static_cast<uint32_t>(std::min(most, T - row)) * d8;
    const size_t at = static_cast<size_t>(row) * d;
    const cudaError_t e = launch_dependent(k_act_dequant, dim3(static_cast<unsigned>(ceil_div(n8, 256 * kDequantSteps))), 256, 0,
                                           1, st, codes + at, sa + row, d8, n8,
                                           static_cast<void*>(static_cast<uint8_t*>(out) + at * (out_bf16 ? 2 : 4)),
                                           static_cast<int>(out_bf16));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qe
