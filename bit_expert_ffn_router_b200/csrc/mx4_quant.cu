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
// leave as one 4-byte word per thread, fp32 values as whole 32-byte sectors
// (two 16-byte stores instead: 205 against 143 us for 98304 x 2048). Four such
// units per thread keep their loads in flight together. 16-bit rows are near
// the issue limit too, so maxima are taken two packed values at a time and rows
// are found with 32-bit arithmetic. 98304 x 2048 fp32: 144 us (6.3 TB/s), and
// back 143 us; bf16 84 us (6.1 TB/s) and 82 us.
#include <string.h>

#include <type_traits>

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQUnits = 4;  // units of 8 values per thread: their loads are in flight together

// Eight values as fp32 and the largest magnitude among them; NaN if one is.
template <typename T>
struct Values;

template <>
struct Values<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = ld_plain(reinterpret_cast<const float4*>(p)), b = ld_plain(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void load_each(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ld_plain(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ float top() const {
    float m = fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = nan_max(m, fabsf(v[i]));
    m = nan_max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return nan_max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  }
  __device__ __forceinline__ static float nan_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  }
};

// 16-bit types stay packed in pairs: magnitudes and their maximum two at a time.
template <typename T2>
struct Pairs {
  uint32_t w[4];
  template <typename T>
  __device__ __forceinline__ void load(const T* p) {
    const uint4 a = ld_plain(reinterpret_cast<const uint4*>(p));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  }
  template <typename T>
  __device__ __forceinline__ void load_each(const T* p) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ld_plain(q + 2 * i) | static_cast<uint32_t>(ld_plain(q + 2 * i + 1)) << 16;
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ static T2 as2(uint32_t x) { return *reinterpret_cast<const T2*>(&x); }
  __device__ __forceinline__ static uint32_t bits(T2 x) { return *reinterpret_cast<const uint32_t*>(&x); }
  __device__ __forceinline__ uint32_t top2() const {
    T2 m = __hmax2_nan(as2(w[0] & 0x7fff7fffu), as2(w[1] & 0x7fff7fffu));
    m = __hmax2_nan(m, __hmax2_nan(as2(w[2] & 0x7fff7fffu), as2(w[3] & 0x7fff7fffu)));
    m = __hmax2_nan(m, as2(__shfl_xor_sync(0xffffffffu, bits(m), 1)));
    m = __hmax2_nan(m, as2(__shfl_xor_sync(0xffffffffu, bits(m), 2)));
    return bits(m);
  }
};
template <>
struct Values<__nv_bfloat16> : Pairs<__nv_bfloat162> {
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ float top() const {
    const uint32_t m = top2();
    return Values<float>::nan_max(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};
template <>
struct Values<__half> : Pairs<__half2> {
  __device__ __forceinline__ float get(int i) const {
    const __half2 h = as2(w[i / 2]);
    return (i & 1) ? __high2float(h) : __low2float(h);
  }
  __device__ __forceinline__ float top() const {
    const __half2 m = as2(top2());
    return Values<float>::nan_max(__low2float(m), __high2float(m));
  }
};

// a * b on two fp32 lanes at once.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
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

// Row (from the CTA's first) and unit (of 8 values) of the CTA's local-th
// unit: one 64-bit division per CTA, then a multiplication by ceil(2^32 / upr),
// exact while n * upr < 2^32 (cols <= kMx4MaxCols: n < upr + 1024 <= 9216).
struct RowOf {
  long long row0;
  uint32_t rem0, upr, magic, count;
  __device__ RowOf(long long units, uint32_t upr_, uint32_t magic_) : upr(upr_), magic(magic_) {
    const long long u0 = static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits);
    row0 = u0 / upr;
    rem0 = static_cast<uint32_t>(u0 - row0 * upr);
    count = static_cast<uint32_t>(min(units - u0, static_cast<long long>(kQThreads * kQUnits)));
  }
  __device__ __forceinline__ void at(uint32_t local, uint32_t& row, uint32_t& unit) const {
    const uint32_t n = rem0 + local;
    row = __umulhi(n, magic);
    unit = n - row * upr;
  }
};

// Rows of x: by single values, in 16-byte loads, or those of one flat array (no
// row to look for before the load; bf16 is near the issue limit).
enum Rows { kSingle, kVector, kFlat };

template <typename T, int ROWS>
__global__ void __launch_bounds__(kQThreads) mx4_quantize_kernel(const T* x, long long ld,
                                                                 long long units, uint32_t upr, uint32_t magic,
                                                                 int pitch, uint8_t* __restrict__ codes,
                                                                 uint8_t* __restrict__ scales) {
  const RowOf rows(units, upr, magic);
  x += ROWS == kFlat ? static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits * 8) : rows.row0 * ld;
  scales += rows.row0 * pitch;
  uint32_t* out = reinterpret_cast<uint32_t*>(codes) + static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits);
  grid_dep_wait();
  // a product that follows sets up meanwhile and waits for this grid's end; what
  // came before this grid has ended by now, so nothing of it is overtaken
  grid_dep_launch();
  Values<T> v[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    const T* p = x + local * 8;
    if (ROWS != kFlat) {
      uint32_t row, unit;
      rows.at(local, row, unit);
      p = x + row * ld + unit * 8;
    }
    if (local >= rows.count)
      v[i].zero();
    else if (ROWS != kSingle)
      v[i].load(p);
    else
      v[i].load_each(p);
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    const float m = v[i].top();
    const bool bad = !(m < INFINITY);
    const uint32_t e = max(static_cast<int>(__float_as_uint(m) >> 23) - 2, 0);
    const float inv = __uint_as_float((254u - e) << 23);
    float s[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 q = fmul2(make_float2(v[i].get(2 * j), v[i].get(2 * j + 1)), make_float2(inv, inv));
      s[2 * j] = q.x, s[2 * j + 1] = q.y;
    }
    const uint32_t c = codes8(s);
    if (local >= rows.count) continue;
    out[local] = bad ? 0u : c;
    if ((threadIdx.x & 3) == 0) {  // the block's first lane: rows are whole blocks
      uint32_t row, unit;
      rows.at(local, row, unit);
      uint8_t* b = scales + row * static_cast<uint32_t>(pitch) + (unit >> 2);
      *b = bad ? 255 : static_cast<uint8_t>(e);
      if (unit + 4 == upr)  // the row's last block also clears the padding
        for (int k = upr / 4; k < pitch; ++k) *++b = 0;
    }
  }
}

// Eight fp32 results to p in T.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const float* v) {
  constexpr int kW = 2 * sizeof(T);
  uint32_t w[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  if (VEC && sizeof(T) == 4) {  // 32 bytes, a whole sector, at once
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[kW - 4]), "r"(w[kW - 3]), "r"(w[kW - 2]), "r"(w[kW - 1])
                 : "memory");
  } else if (VEC) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    T o[8];
    memcpy(o, w, sizeof(o));
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = o[j];
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQThreads) mx4_dequantize_kernel(const uint8_t* codes,
                                                                   const uint8_t* scales,
                                                                   long long units, uint32_t upr, uint32_t magic,
                                                                   int pitch, T* __restrict__ out, long long ld) {
  const RowOf rows(units, upr, magic);
  out += rows.row0 * ld;
  scales += rows.row0 * pitch;
  const uint32_t* in = reinterpret_cast<const uint32_t*>(codes) + static_cast<long long>(blockIdx.x) * (kQThreads * kQUnits);
  grid_dep_wait();  // and no early launch of the next: what is written here may be anything
  uint32_t c[kQUnits], s[kQUnits];
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    uint32_t row, unit;
    rows.at(local, row, unit);
    if (local < rows.count) {
      c[i] = ld_plain(in + local);
      s[i] = ld_plain(scales + row * pitch + (unit >> 2));
    }
  }
#pragma unroll
  for (int i = 0; i < kQUnits; ++i) {
    const uint32_t local = i * kQThreads + threadIdx.x;
    if (local >= rows.count) continue;
    uint32_t row, unit;
    rows.at(local, row, unit);
    // 2^(s - 127): s = 0 is the subnormal 2^-127, s = 255 is NaN
    const float f = __uint_as_float(s[i] == 0 ? 0x00400000u : s[i] == 255 ? 0x7fffffffu : s[i] << 23);
    float v[8];
    levels8(c[i], v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 q = fmul2(make_float2(v[2 * j], v[2 * j + 1]), make_float2(f, f));
      v[2 * j] = q.x, v[2 * j + 1] = q.y;
    }
    store8<T, VEC>(out + row * ld + unit * 8, v);
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

// Whether every row starts on `align` bytes.
bool vec_ok(const void* p, size_t row_bytes, size_t align) {
  return reinterpret_cast<uintptr_t>(p) % align == 0 && row_bytes % align == 0;
}

template <typename T>
cudaError_t quantize(const void* x, int rows, int cols, size_t ld, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const Units u = units_of(rows, cols);
  const T* p = static_cast<const T*>(x);
  const int pitch = mx4_pitch(cols);
  const bool vec = vec_ok(x, ld * sizeof(T), 16);
  return launch_dependent(!vec                                 ? mx4_quantize_kernel<T, kSingle>
                          : ld == static_cast<size_t>(cols) ? mx4_quantize_kernel<T, kFlat>
                                                            : mx4_quantize_kernel<T, kVector>,
                          u.grid, kQThreads, 0, s, p, ld, u.units, u.upr, u.magic, pitch, codes, scales);
}

template <typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, int rows, int cols, void* out, size_t ld,
                       cudaStream_t s) {
  const Units u = units_of(rows, cols);
  T* p = static_cast<T*>(out);
  const int pitch = mx4_pitch(cols);
  return launch_dependent(
      vec_ok(out, ld * sizeof(T), 8 * sizeof(T)) ? mx4_dequantize_kernel<T, true> : mx4_dequantize_kernel<T, false>, u.grid,
      kQThreads, 0, s, codes, scales, u.units, u.upr, u.magic, pitch, p, ld);
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
