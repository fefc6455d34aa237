// Quantization arithmetic shared by the kernels that write activation codes: bf16 conversion, the
// symmetric integer codes (A6/A8, W4/W3) and the MXFP4 block (E2M1 codes, E8M0 scale).
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace qe {

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16_bits(float v) {
  __nv_bfloat16 h = __float2bfloat16_rn(v);
  return *reinterpret_cast<uint16_t*>(&h);
}

// One symmetric RTN code: clamp(rint(fl32(v / scale)), -qmax, qmax); zero scale -> 0.
__device__ __forceinline__ int rtn_code(float v, float scale, int qmax) {
  if (scale == 0.0f) return 0;
  float r = rintf(__fdiv_rn(v, scale));
  r = fminf(fmaxf(r, -static_cast<float>(qmax)), static_cast<float>(qmax));
  return static_cast<int>(r);
}

// Eight codes through rtn_code, packed little-endian into two words. Kept out of line: callers
// unroll their loops, and this rare path would otherwise be copied into every unrolled step.
static __device__ __noinline__ uint2 rtn_code8_exact(float v0, float v1, float v2, float v3, float v4, float v5, float v6,
                                              float v7, float scale, int qmax) {
  const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  uint32_t w0 = 0, w1 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w0 |= (static_cast<uint32_t>(rtn_code(v[i], scale, qmax)) & 0xFFu) << (8 * i);
    w1 |= (static_cast<uint32_t>(rtn_code(v[4 + i], scale, qmax)) & 0xFFu) << (8 * i);
  }
  return make_uint2(w0, w1);
}

// Eight codes rtn_code(v[i], scale, qmax), packed little-endian into two words, without a division
// in the common case. inv = fl32(1/scale), the correctly rounded reciprocal. g = fl32(v*inv) differs
// from the correctly rounded quotient fl32(v/scale) by at most 3 units of 2^-24 |g|, so rint(g)
// equals rint(fl32(v/scale)) unless g lies within that distance of a half-integer; the test below
// asks for a margin of 2^-20 |g| and sends the rest through rtn_code. The fast path also needs a
// normal scale, and |g| < qmax + 0.5 so that the clamp does not bind (|v| <= absmax keeps
// |g| <= qmax (1 + 2^-22) when the scale came from this row's absmax).
// rint uses the 1.5*2^23 trick: fl32(g + 1.5*2^23) holds rint(g) (half to even) in its low bits.
__device__ __forceinline__ void rtn_code8(const float (&v)[8], float scale, float inv, bool fast, int qmax,
                                          uint32_t& w0, uint32_t& w1) {
  constexpr float kM = 12582912.0f;
  const float qmax_f = static_cast<float>(qmax) + 0.5f;
  uint32_t b[8];
  bool ok = fast;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = __fmul_rn(v[i], inv);
    const float t = __fadd_rn(g, kM);
    const float d = fabsf(__fsub_rn(g, __fsub_rn(t, kM)));
    ok = ok && (__fmaf_rn(fabsf(g), 9.5367431640625e-07f, d) < 0.5f) && (fabsf(g) < qmax_f);
    b[i] = __float_as_uint(t);
  }
  if (ok) {
    w0 = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    w1 = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return;
  }
  const uint2 w = rtn_code8_exact(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], scale, qmax);
  w0 = w.x;
  w1 = w.y;
}
// Whether rtn_code8's fast path may be used for this scale (and its reciprocal).
__device__ __forceinline__ bool rtn_fast_ok(float scale, float inv) {
  return scale >= 1.17549435e-38f && inv < 3.0e38f;
}

// ------------------------------------------------------------------ MXFP4
// 32 consecutive channels of a row share a scale 2^E, stored as the byte E + 127 (E8M0); the codes are
// E2M1 (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6). E = floor(log2 max|v|) - 2
// puts the largest magnitude into [4, 8), the top binade of E2M1, where it saturates at 6; E is kept in
// [-127, 127]. A block that holds a NaN or an infinity gets the byte 255 (NaN) and codes 0, so that it
// stays visible in whatever is computed from it.
constexpr int kMxBlock = 32;
constexpr int kMxTileRows = 128;   // rows and
constexpr int kMxTileCols = 128;   // channels of a tile of scale bytes (512 bytes)
constexpr int kMxTileBytes = 512;
constexpr uint32_t kMxOne = 127u;  // a scale of one: what blocks past a row's end hold

// Byte offset of row r's four scales in the first of its KT = ceil(cols / 128) tiles; those of channels
// [128*kt, 128*kt + 128) are kt * 512 bytes on. The order inside a tile is the one tcgen05.cp 32x128b
// spreads over the tensor memory lanes: 16 bytes for each row r % 32, four for each r / 32.
__host__ __device__ __forceinline__ size_t mx_scale_row(size_t r, size_t KT) {
  return (r >> 7) * KT * kMxTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}
// Offset of channel k's scale from there.
__host__ __device__ __forceinline__ int mx_scale_at(int k) {
  return (k / kMxTileCols) * kMxTileBytes + k % kMxTileCols / kMxBlock;
}

// Scale byte of a block whose largest |v| has the bits `top` (fp32, sign cleared).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int e = static_cast<int>(top >> 23) - 2;  // (field - 127) - 2 + 127; subnormals clamp below
  return static_cast<uint32_t>(e > 0 ? e : 0);
}
// 2^-E for a scale byte below 255 (E in [-127, 125], so the factor is a normal number).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^E of a scale byte; NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// Eight E2M1 codes of a[i], ties to even, saturating at 6; code i in bits [4i, 4i+4).
__device__ __forceinline__ uint32_t e2m1_pack8(const float (&a)[8]) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
  return w;
}

// The bits of max |v[i]|; those of a NaN (0x7FFFFFFF, above infinity's) when one is among them.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8]) {
  float m = max3_abs(v[0], v[1], v[2]);
  m = max3_abs(m, v[3], v[4]);
  m = max3_abs(m, v[5], v[6]);
  return __float_as_uint(max3_abs(m, v[7], v[7]));
}

// a[i] * b[i], a[i] * x and a[i] + x, two per instruction (each one IEEE operation).
__device__ __forceinline__ void mul8(float (&a)[8], const float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a[i]), "+f"(a[i + 1])
        : "f"(b[i]), "f"(b[i + 1]));
}
__device__ __forceinline__ void mul8(float (&a)[8], float x) {
  const float b[8] = {x, x, x, x, x, x, x, x};
  mul8(a, b);
}

// Codes of eight values of a block whose scale byte is `byte`. v * 2^-E is exact unless it falls below
// fp32's normal range, where the code is 0 either way.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8], uint32_t byte) {
  float a[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  mul8(a, mx_inv_scale(byte));
  const uint32_t code = e2m1_pack8(a);
  return byte == 255u ? 0u : code;
}

// rtn_code8 for a row whose scale came from its own finite absmax, so that g = fl32(v * inv) has |g| <= qmax (1 + 2^-22)
// and the clamp cannot bind. g is off the correctly rounded quotient by at most 3 * 2^-24 |g|, below
// (qmax + 1) * 2^-22, so rint(g) is the code when its distance to g stays below limit = 0.5 - (qmax + 1) * 2^-22.
__device__ __forceinline__ float rtn_limit(int qmax) {
  return 0.5f - static_cast<float>(qmax + 1) * 2.384185791015625e-07f;
}
__device__ __forceinline__ void rtn_code8_row(const float (&v)[8], float scale, float inv, float limit, int qmax,
                                              uint32_t& w0, uint32_t& w1) {
  uint32_t b[8];
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float t0, t1;
    asm("{\n\t.reg .b64 g, t, r, k;\n\t"
        "mov.b64 g, {%4, %5};\n\tmov.b64 k, {%6, %6};\n\tmul.rn.f32x2 g, g, k;\n\t"
        "mov.b64 k, {0f4B400000, 0f4B400000};\n\tadd.rn.f32x2 t, g, k;\n\t"
        "mov.b64 k, {0fCB400000, 0fCB400000};\n\tadd.rn.f32x2 r, t, k;\n\t"
        "mov.b64 k, {0fBF800000, 0fBF800000};\n\tfma.rn.f32x2 g, r, k, g;\n\t"
        "mov.b64 {%0, %1}, t;\n\tmov.b64 {%2, %3}, g;\n\t}"
        : "=f"(t0), "=f"(t1), "=f"(d[i]), "=f"(d[i + 1])
        : "f"(v[i]), "f"(v[i + 1]), "f"(inv));
    b[i] = __float_as_uint(t0);
    b[i + 1] = __float_as_uint(t1);
  }
  if (absmax8(d) < __float_as_uint(limit)) {
    w0 = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    w1 = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return;
  }
  const uint2 w = rtn_code8_exact(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], scale, qmax);
  w0 = w.x;
  w1 = w.y;
}

// Two fp32 values as a word of bf16 (the first in the low half).
__device__ __forceinline__ uint32_t bf16x2_word(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace qe
