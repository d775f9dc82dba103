// Rows to microscaled 4-bit floating point (the MX format with 4-bit
// elements) and back.
//
// A row is cut into blocks of 32 values. With m = max |v| over a block,
//   e    = clamp(floor(log2 m) - 2, -127, 127)   (2 = exponent of the largest
//                                                 level, 6 = 1.5 * 2^2)
//   q_i  = v_i / 2^e rounded to the levels 0, .5, 1, 1.5, 2, 3, 4, 6 (nearest,
//          ties to the level with an even last bit; above 6: 6), sign kept
// and the stored bytes are e + 127 per block and two q per byte. In the bits
// of an fp32 m, e + 127 is simply max(exponent field - 2, 0): a subnormal m
// has field 0, and the largest finite one gives 252. 2^-e is then the fp32
// number with the exponent field 254 - (e + 127), so v / 2^e is one exact
// multiplication (inexact only where the product is subnormal, far below the
// first rounding border 0.25). bf16 and fp16 convert to fp32 exactly.
//
// Both directions only move bytes, and the byte counts are the bound: each
// thread takes 8 values of a row (one 16-byte load of 16-bit values, two of
// fp32), a block's maximum takes two shuffles among its four lanes, the codes
// leave as one 4-byte word per thread.
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQUnits = 4;  // units of 8 values per thread: their loads are in flight together

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float* v);

template <>
__device__ __forceinline__ void load8<float, true>(const float* p, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16, true>(const __nv_bfloat16* p, float* v) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half, true>(const __half* p, float* v) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, float* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(p[i]);
}

// Eight values to eight codes, value 0 in the lowest four bits.
__device__ __forceinline__ uint32_t codes8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes to the fp32 levels they name.
__device__ __forceinline__ void levels8(uint32_t c, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Row and unit (8 values) of a flat unit index, from the index of the CTA's
// first unit: one 64-bit division per CTA, then a multiplication by
// ceil(2^32 / upr), exact while n * upr < 2^32 (cols <= kMx4MaxCols: n < upr +
// 1024 <= 9216).
struct RowOf {
  long long row0;
  uint32_t rem0, upr, magic;
  __device__ RowOf(long long u0, uint32_t upr_, uint32_t magic_) : upr(upr_), magic(magic_) {
    row0 = u0 / upr;
    rem0 = static_cast<uint32_t>(u0 - row0 * upr);
  }
  __device__ __forceinline__ void at(uint32_t local, long long& row, uint32_t& unit) const {
    const uint32_t n = rem0 + local;
    const uint32_t q = __umulhi(n, magic);
    row = row0 + q;
    unit = n - q * upr;
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) mx4_quantize_kernel(const T* __restrict__ x, long long ld,
                                                                 long long units, uint32_t upr, uint32_t magic,
                                                                 int pitch, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  const long long u0 = static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits);
  const RowOf rows(u0, upr, magic);
  grid_dep_launch();  // a product that follows sets up meanwhile; it waits for this grid's end
  grid_dep_wait();
  float v[kQUnits][8];
  long long row[kQUnits];
  uint32_t unit[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    rows.at(local, row[i], unit[i]);
    if (u0 + local < units) {
      load8<T, VEC>(x + row[i] * ld + unit[i] * 8, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    // magnitudes compare as integers; infinities and NaN come out on top
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const bool bad = m >= 0x7f800000u;
    const int e = max(static_cast<int>(m >> 23) - 2, 0);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= inv;
    const uint32_t c = bad ? 0u : codes8(v[i]);
    if (u0 + local >= units) continue;
    *reinterpret_cast<uint32_t*>(codes + (u0 + local) * 4) = c;
    if ((unit[i] & 3) == 0) {
      uint8_t* s = scales + row[i] * pitch + (unit[i] >> 2);
      *s = bad ? 255 : static_cast<uint8_t>(e);
      if (unit[i] + 4 == upr)  // the row's last block also clears the padding
        for (int b = upr / 4; b < pitch; ++b) scales[row[i] * pitch + b] = 0;
    }
  }
}

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) mx4_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales,
                                                                   long long units, uint32_t upr, uint32_t magic,
                                                                   int pitch, T* __restrict__ out, long long ld) {
  const long long u0 = static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits);
  const RowOf rows(u0, upr, magic);
  grid_dep_launch();  // a product that follows sets up meanwhile; it waits for this grid's end
  grid_dep_wait();
  uint32_t c[kQUnits], s[kQUnits];
  long long row[kQUnits];
  uint32_t unit[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    rows.at(local, row[i], unit[i]);
    if (u0 + local < units) {
      c[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (u0 + local) * 4));
      s[i] = __ldg(scales + row[i] * pitch + (unit[i] >> 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    if (u0 + i * kQThreads + threadIdx.x >= units) continue;
    // 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 is NaN
    const float f = __uint_as_float(s[i] == 0 ? 0x00400000u : s[i] == 255 ? 0x7fffffffu : s[i] << 23);
    float v[8];
    levels8(c[i], v);
    T o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = from_f32<T>(v[j] * f);
    T* p = out + row[i] * ld + unit[i] * 8;
    if (VEC) {
#pragma unroll
      for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j)
        reinterpret_cast<uint4*>(p)[j] = reinterpret_cast<const uint4*>(o)[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = o[j];
    }
  }
}

struct Units {
  long long units;
  uint32_t upr, magic;
  unsigned grid;
};

Units units_of(int rows, int cols) {
  Units u;
  u.upr = static_cast<uint32_t>(cols / 8);
  u.units = static_cast<long long>(rows) * u.upr;
  u.magic = static_cast<uint32_t>(((1ull << 32) + u.upr - 1) / u.upr);
  u.grid = static_cast<unsigned>((u.units + kQThreads * kQUnits - 1) / (kQThreads * kQUnits));
  return u;
}

bool vec_ok(const void* p, size_t ld, size_t size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * size) % 16 == 0;
}

template <typename T>
cudaError_t quantize(const void* x, int rows, int cols, size_t ld, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const Units u = units_of(rows, cols);
  const T* p = static_cast<const T*>(x);
  const int pitch = mx4_pitch(cols);
  if (vec_ok(x, ld, sizeof(T)))
    return launch_dependent(mx4_quantize_kernel<T, true>, u.grid, kQThreads, 0, s, p, ld, u.units, u.upr, u.magic, pitch,
                            codes, scales);
  return launch_dependent(mx4_quantize_kernel<T, false>, u.grid, kQThreads, 0, s, p, ld, u.units, u.upr, u.magic, pitch,
                          codes, scales);
}

template <typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out, size_t ld,
                       cudaStream_t s) {
  const Units u = units_of(rows, cols);
  T* p = static_cast<T*>(out);
  const int pitch = mx4_pitch(cols);
  if (vec_ok(out, ld, sizeof(T)))
    return launch_dependent(mx4_dequantize_kernel<T, true>, u.grid, kQThreads, 0, s, codes, scales, u.units, u.upr, u.magic, pitch,
                            p, ld);
  return launch_dependent(mx4_dequantize_kernel<T, false>, u.grid, kQThreads, 0, s, codes, scales, u.units, u.upr, u.magic, pitch,
                          p, ld);
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int type, int rows, int cols, size_t ld, uint8_t* codes,
                                uint8_t* scales, cudaStream_t s) {
  if (type == MOE_TYPE_BF16) return quantize<__nv_bfloat16>(x, rows, cols, ld, codes, scales, s);
  if (type == MOE_TYPE_FP16) return quantize<__half>(x, rows, cols, ld, codes, scales, s);
  return quantize<float>(x, rows, cols, ld, codes, scales, s);
}

cudaError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out, int type,
                                  size_t ld, cudaStream_t s) {
  if (type == MOE_TYPE_BF16) return dequantize<__nv_bfloat16>(codes, scales, rows, cols, out, ld, s);
  if (type == MOE_TYPE_FP16) return dequantize<__half>(codes, scales, rows, cols, out, ld, s);
  return dequantize<float>(codes, scales, rows, cols, out, ld, s);
}

}  // namespace moe
