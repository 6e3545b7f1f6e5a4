// Microscaled formats on the device: eight consecutive values of a thread into elements and the scales of their blocks,
// and back (eagle_mx).
#pragma once
#include <cuda_fp8.h>

#include "internal.h"
#include "common.cuh"

namespace eagle {

// A matrix's addresses as kernels take them.
struct MxView {
  uint8_t* data;
  uint8_t* scale;
  const float* g;          // tensor factor, null: 1
  int rows, cols;
  int groups;              // 4-scale groups of a row
};

inline MxView mx_view(const eagle_mx* m) {
  MxView v;
  v.data = static_cast<uint8_t*>(m->data);
  v.scale = m->scale;
  v.g = m->format == EAGLE_NV_FP4 ? m->tensor_scale : nullptr;
  v.rows = m->rows;
  v.cols = m->cols;
  v.groups = (m->cols / (m->format == EAGLE_NV_FP4 ? 16 : 32) + 3) / 4;
  return v;
}

template <int FMT>
constexpr int mx_block() { return FMT == EAGLE_NV_FP4 ? 16 : 32; }

// Byte of scale 4 c of row r.
__device__ __forceinline__ size_t mx_scale_at(const MxView& m, int r, int c) {
  return (static_cast<size_t>(r >> 7) * m.groups + c) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

__device__ __forceinline__ float mx_decode_e4m3(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ uint32_t mx_pack_e2m1(const float (&v)[8]) {
  uint32_t w;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}
__device__ __forceinline__ uint32_t mx_pack_e4m3(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
      " mov.b32 %0, {l, h};\n}\n"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

__device__ __forceinline__ float mx_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Divisors under which a Newton step's remainder may have bits below fp32's smallest number, 2^-149 (a quotient's last bit
// times the divisor's: from 2^-10 on, the smallest border of a scale, 2^-33 2^-23 d), so that near a border the quotient would
// not be the rounded one; above the inverse of it the inverse loses its own.  There a scale's quotient is a division, and
// elements and their divisor are taken 2^64 times larger.
constexpr float MX_SMALL = 0x1p-80f;

// The tensor's factor as quantisations take it: 6 g and its inverse, infinite where quotients are divisions.
struct MxFactor {
  float g, g6, r6;
};
__device__ __forceinline__ MxFactor mx_factor(const MxView& m) {
  MxFactor f;
  f.g = m.g ? *m.g : 1.0f;
  f.g6 = 6.0f * f.g;
  f.r6 = f.g6 >= MX_SMALL && f.g6 <= 1.0f / MX_SMALL ? 1.0f / f.g6 : INFINITY;
  return f;
}

// The fp32 quotient x / d, given r = 1 / d to a step or two: one Newton step on x r (Markstein 1990: the remainder x - q d is
// exact in one fused operation), so that a quotient that fp32 has, a tie among them, is met exactly.
__device__ __forceinline__ float mx_quotient(float x, float d, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, d, x), r, q);
}

// Eight consecutive values of row `row` from column `col` (a multiple of 8) on, held by each lane of a warp for
// consecutive columns from a multiple of 256 on: elements, and the scales of their blocks.  Lanes past the last column
// (`in` false) hold zeros.  Returns whether the block has a NaN or an infinity.
template <int FMT>
__device__ __forceinline__ bool mx_put(const MxView& m, const MxFactor& f, int row, int col, bool in, const float (&x)[8],
                                       int lane) {
  float most = fabsf(x[0]);                      // NaN if any is
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(fabsf(x[i])));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(__shfl_xor_sync(0xffffffffu, most, 1)));
  if (FMT != EAGLE_NV_FP4) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(__shfl_xor_sync(0xffffffffu, most, 2)));
  const uint32_t top = __float_as_uint(most);
  const bool bad = top >= 0x7f800000u;
  uint32_t byte;
  float v[8];
  if (FMT == EAGLE_NV_FP4) {
    // (a quotient beyond the type's range saturates: it is held where its remainder stays finite)
    const float q = fminf(most * f.r6, 1e6f);
    const float t = f.r6 < INFINITY ? fmaf(fmaf(-q, f.g6, most), f.r6, q) : most / f.g6;
    byte = bad ? 0x7fu
           : top == 0u ? 0u
                       : static_cast<uint32_t>(__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3));
    const float d = mx_decode_e4m3(byte) * f.g;
    const float r = d >= 0x1p-126f ? mx_rcp(d) : 0.0f;
    // elements far beyond 6, whose remainder may not be finite, and small divisors
    if (__any_sync(0xffffffffu, fmaxf(most, 1e30f * MX_SMALL) * r > 1e30f)) {
      const bool small = r > 1.0f / MX_SMALL;
      const float up = small ? 0x1p64f : 1.0f, down = small ? 0x1p-64f : 1.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = fabsf(x[i] * r) < 16.0f ? mx_quotient(x[i] * up, d * up, r * down) : x[i] * r;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = mx_quotient(x[i], d, r);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = copysignf(v[i], x[i]);   // (a zero keeps its sign)
  } else {
    // the largest element is 1.75 * 2^8 (e4m3) or 1.5 * 2^2 (e2m1); a power of two and its inverse are exact
    const uint32_t lead = FMT == EAGLE_MX_FP8 ? 0x600000u : 0x400000u;
    const int whole = FMT == EAGLE_MX_FP8 ? 8 : 2;
    const int e = static_cast<int>(top >> 23) - whole + ((top & 0x7fffffu) > lead ? 1 : 0);
    byte = bad ? 255u : static_cast<uint32_t>(max(e, 0));
    const float inv = __uint_as_float(bad ? 0x7fffffffu : (254u - byte) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i] * inv;
  }
  const int shift = FMT == EAGLE_NV_FP4 ? 1 : 2;                 // lanes a block, as a power of two
  uint32_t word = byte << (8 * ((lane >> shift) & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 1 << shift);
  word |= __shfl_xor_sync(0xffffffffu, word, 2 << shift);
  if (in) {
    if (FMT == EAGLE_MX_FP8) {
      *reinterpret_cast<uint2*>(m.data + static_cast<size_t>(row) * m.cols + col) =
          make_uint2(mx_pack_e4m3(v[0], v[1], v[2], v[3]), mx_pack_e4m3(v[4], v[5], v[6], v[7]));
    } else {
      *reinterpret_cast<uint32_t*>(m.data + (static_cast<size_t>(row) * m.cols + col) / 2) = mx_pack_e2m1(v);
    }
    if ((lane & ((4 << shift) - 1)) == 0)
      *reinterpret_cast<uint32_t*>(m.scale + mx_scale_at(m, row, col / (4 * mx_block<FMT>()))) = word;
  }
  return bad && in;
}

// Eight elements of a row from `col` on and their scale as they lie in memory, and their values.
template <int FMT>
struct MxRaw {
  uint2 w;                 // (4 bits: the first word)
  uint32_t byte;
  __device__ __forceinline__ void load(const MxView& m, int row, int col) {
    const int block = col / mx_block<FMT>();
    byte = m.scale[mx_scale_at(m, row, block >> 2) + (block & 3)];
    const size_t at = static_cast<size_t>(row) * m.cols + col;
    if (FMT == EAGLE_MX_FP8) w = *reinterpret_cast<const uint2*>(m.data + at);
    else w.x = *reinterpret_cast<const uint32_t*>(m.data + at / 2);
  }
};
template <int FMT>
__device__ __forceinline__ void mx_get(const MxRaw<FMT>& raw, float g, float (&v)[8]) {
  const uint32_t byte = raw.byte;
  float d;
  if (FMT == EAGLE_NV_FP4) d = mx_decode_e4m3(byte) * g;
  else d = __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 1u << 22 : byte << 23);
  if (FMT == EAGLE_MX_FP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t two = ((i < 2 ? raw.w.x : raw.w.y) >> (16 * (i & 1))) & 0xffffu;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      v[2 * i] = f.x * d;
      v[2 * i + 1] = f.y * d;
    }
  } else {
    const uint32_t w = raw.w.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // sign, two bits of exponent (bias 1) and one of fraction, as a float 2^126 times too small
      const uint32_t c = w >> (4 * i);
      const float f = __uint_as_float(((c & 8u) << 28) | ((c & 7u) << 22)) * 0x1p126f;
      v[i] = f * d;
    }
  }
}

// Eight elements of a row as they lie in memory, and their values.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uint4 w;
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  Raw8<T> r;
  r.load(p);
  r.get(x);
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace eagle
