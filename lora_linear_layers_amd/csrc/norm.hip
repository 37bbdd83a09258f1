// norm.hip - what stands between a block's residual stream and its
// projections: the root-mean-square norm with the residual's addition, its
// gradient, and rows kept in 8 bits (the norm's output, or any activation),
// plus their host-side launchers (internal interface in launch.h).
//
//     h = x + residual (rounded to the type),  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd w
//
// All of them are streams of rows: each row is read once into registers, its
// statistics are formed there, and it is written from there, so what bounds
// them is the memory's rate or, for a few rows, the launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"

namespace lora {

namespace {

// A row belongs to TPR threads of a block (16: four rows a wave; 64: a wave;
// 256, 1024: a block); each holds NV chunks of 8 elements.  VEC: rows of whole
// aligned chunks, chunk k of thread t at element 8 (TPR k + t), in 16-byte
// accesses; else element e of chunk k at TPR (8 k + e) + t, one by one.
template <int TPR, int NV, bool VEC>
struct Row {
  static constexpr int NT = TPR < 256 ? 256 : TPR;  // threads of a block
  static constexpr int RPB = NT / TPR;              // rows of a block
  static __device__ __forceinline__ int col(int t, int k, int e) { return VEC ? 8 * (TPR * k + t) + e : TPR * (8 * k + e) + t; }
};

// The 8 elements of chunk k as floats (0 past d).
template <typename T, int TPR, int NV, bool VEC>
__device__ __forceinline__ void get8(const T* row, int d, int t, int k, float (&f)[8]) {
  using R = Row<TPR, NV, VEC>;
  if constexpr (VEC) {
    const int c = R::col(t, k, 0);
    if constexpr (sizeof(T) == 2) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (c < d) v = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = __builtin_bit_cast(float, v[q] << 16);
        f[2 * q + 1] = __builtin_bit_cast(float, v[q] & 0xFFFF0000u);
      }
    } else {
      f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
      if (c < d) {
        a = *reinterpret_cast<const f32x4*>(row + c);
        b = *reinterpret_cast<const f32x4*>(row + c + 4);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[q] = a[q];
        f[4 + q] = b[q];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = R::col(t, k, e);
      f[e] = 0.f;
      if (c < d) {
        if constexpr (sizeof(T) == 2)
          f[e] = __builtin_bit_cast(float, (uint32_t)row[c] << 16);
        else
          f[e] = row[c];
      }
    }
  }
}

template <typename T, int TPR, int NV, bool VEC>
__device__ __forceinline__ void put8(T* row, int d, int t, int k, const float (&f)[8]) {
  using R = Row<TPR, NV, VEC>;
  if constexpr (VEC) {
    const int c = R::col(t, k, 0);
    if (c >= d) return;
    if constexpr (sizeof(T) == 2) {
      u32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
      *reinterpret_cast<u32x4*>(row + c) = v;
    } else {
      *reinterpret_cast<f32x4*>(row + c) = f32x4{f[0], f[1], f[2], f[3]};
      *reinterpret_cast<f32x4*>(row + c + 4) = f32x4{f[4], f[5], f[6], f[7]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = R::col(t, k, e);
      if (c < d) store_out<T>(row, c, f[e]);
    }
  }
}

// What the type holds of a float.
template <typename T>
__device__ __forceinline__ float rounded(float x) {
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(float, (uint32_t)f2bf(x) << 16);
  else
    return x;
}

// The sum (or maximum) over a row's threads, in a fixed order.  red: NT / 64
// floats of LDS, one use of them at a time.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_join(float v, float* red) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o));
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // (the last use of red is over)
    if ((threadIdx.x & 63) == 0) red[w] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int q = 1; q < TPR / 64; ++q) v = op(v, red[q]);
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ double row_join64(double v, double* red) {
  constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (TPR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int q = 1; q < TPR / 64; ++q) v += red[q];
  }
  return v;
}

__device__ __forceinline__ bool finite(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u; }

// The power of two a row is kept at: the smallest 2^e, e >= -126, with
// top 2^-e <= 448 (1 for a row of zeros).  top = m 2^k, 1 <= m < 2, and 448 is
// 1.75 2^8: e = k - 8, or k - 7 where m > 1.75.  e4m3 is a floating type, so a
// power of two costs no precision, and an e4m3 code times it is a bf16 number, but for the
// smallest codes at 2^-126 and 2^-125 (bf16 has steps of 2^-133 there) and 256 at 2^120 (2^128:
// a value of 1.9375 2^127 or more, which rounds up to it, comes back infinite).
__device__ __forceinline__ int pack_exponent(float top) {
  const uint32_t b = __builtin_bit_cast(uint32_t, top);
  if (b == 0u) return 0;
  return max((int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
}
__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// Four values (|v| <= 448, or NaN for one that was not finite) as e4m3 codes.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// The nearest float to v on the odd side: where v lies between two floats, the one
// with the odd last bit.  Rounded again to fewer bits, it gives what v itself would.
// (An infinity past the range: as y is there, a value that has no code.)
__device__ __forceinline__ float to_odd(double v) {
  const float f = (float)v;
  if (!finite(f)) return f;
  const double g = f;
  uint32_t b = __builtin_bit_cast(uint32_t, f);
  if (g != v && !(b & 1u)) b += fabs(v) > fabs(g) ? 1u : 0xFFFFFFFFu;
  return __builtin_bit_cast(float, b);
}

// The row's codes and scale from its values y.  NEAR: y is off by less than 2^-18
// of itself; where that could decide a code or the scale, exact(k, y8) gives the
// 8 values of chunk k in 64 bits, which then do (a chunk in some thousands).
template <int TPR, int NV, bool VEC, bool NEAR, class F>
__device__ __forceinline__ void pack_row(const float (&y)[NV][8], int d, int t, uint8_t* codes, float* scale, float* red, F exact) {
  using R = Row<TPR, NV, VEC>;
  constexpr float REL = 3.814697265625e-06f;  // 2^-18
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, finite(y[k][e]) ? fabsf(y[k][e]) : 0.f);
  top = row_join<TPR, true>(top, red);
  bool border = false;
  if constexpr (NEAR) {
    border = pack_exponent(top * (1.f + REL)) != pack_exponent(top * (1.f - REL));
    if (border) {  // (of the whole row)
      top = 0.f;
#pragma unroll 1
      for (int k = 0; k < NV; ++k) {
        double v[8];
        exact(k, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float o = fabsf(to_odd(v[e]));
          top = fmaxf(top, finite(o) ? o : 0.f);
        }
      }
      top = row_join<TPR, true>(top, red);
    }
  }
  const int ex = pack_exponent(top);
  const float inv = pow2(-ex);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = finite(y[k][e]) ? y[k][e] * inv : __builtin_nanf("");
    u32x2 v = {codes4(u[0], u[1], u[2], u[3]), codes4(u[4], u[5], u[6], u[7])};
    if constexpr (NEAR) {
      constexpr float UP = 1.f + REL, DN = 1.f - REL;
      const uint32_t a = codes4(u[0] * UP, u[1] * UP, u[2] * UP, u[3] * UP) ^ codes4(u[0] * DN, u[1] * DN, u[2] * DN, u[3] * DN);
      const uint32_t b = codes4(u[4] * UP, u[5] * UP, u[6] * UP, u[7] * UP) ^ codes4(u[4] * DN, u[5] * DN, u[6] * DN, u[7] * DN);
      if (a | b) {
        double w[8];
        exact(k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = finite(y[k][e]) ? to_odd(w[e] * (double)inv) : __builtin_nanf("");
        v = u32x2{codes4(u[0], u[1], u[2], u[3]), codes4(u[4], u[5], u[6], u[7])};
      }
    }
    if constexpr (VEC) {
      const int c = R::col(t, k, 0);
      if (c < d) *reinterpret_cast<u32x2*>(codes + c) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = R::col(t, k, e);
        if (c < d) codes[c] = (uint8_t)(v[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
  if (t == 0) *scale = pow2(ex);
}

// 1 / sqrt(s), s >= 0: of s 4^-k in [1, 4) in 32 bits, then one Newton step (squares
// of bf16 numbers leave fp32's range at 2^64; 0 gives an infinity, an infinity 0).
__device__ __forceinline__ double rsqrt64(double s) {
  const int64_t b = __builtin_bit_cast(int64_t, s);
  const int e = (int)(b >> 52) - 1023, k2 = e & ~1;
  if (e <= -1023 || e == 1024) return 1.f / sqrtf((float)s);
  const double m = __builtin_bit_cast(double, b - ((int64_t)k2 << 52));
  const double r = 1.f / sqrtf((float)m);
  const double r1 = r * (1.5 - 0.5 * m * r * r);
  return __builtin_bit_cast(double, __builtin_bit_cast(int64_t, r1) - ((int64_t)(k2 / 2) << 52));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// The sum of squares is kept in 64 bits (an instruction an element).  PACK: the codes
// are those of the row's exact values: one whose code 32 bits leave open is formed
// in 64 again (pack_row).  (From 32 bits alone a few codes in a million are the
// neighbour's.)
// A row lives in registers between its one read and its writes (but see below); a block is a
// row of more than 1024 elements, or several rows below, so that 16 to 32 bytes a thread and
// input are in flight on every CU.  8192 x 4096 bf16, residual, Y and codes: 302 MB in
// 50 us, 6 TB/s, what reads and writes of this mix reach; 65536 x 128: 34 MB in 10 us;
// 16 x 4096: 3.8 us, the launch.  Odd widths take one element at a time: 2047 x 1001 fp32,
// 35 MB (out of the caches) in 17 us.
// With codes, rows of 4097 to 8192 and of more than 16384 elements (NV = 4) lie in scratch
// memory instead: the border case of pack_row picks a chunk of h by a number that is
// not a constant, which takes h out of the registers on every row.  8192 x 5120 bf16 with
// residual 230 us (60 without codes), 4096 x 8192 137 (42), 2048 x 32768 270 (104).
template <typename T, int TPR, int NV, bool VEC, bool PACK>
__global__ void __launch_bounds__((Row<TPR, NV, VEC>::NT)) rmsnorm_kernel(const RmsNormArgs a) {
  using R = Row<TPR, NV, VEC>;
  __shared__ float red[16];
  __shared__ double red64[16];
  const int t = threadIdx.x % TPR;
  const int64_t row0 = (int64_t)blockIdx.x * R::RPB + threadIdx.x / TPR;
  if (TPR < 256 && row0 >= a.M) return;  // (rows of a wave's part: nothing of the block is waited for)
  const int d = a.d;
  float h[NV][8];
  const T* x = reinterpret_cast<const T*>(a.X) + row0 * a.ldx;
#pragma unroll
  for (int k = 0; k < NV; ++k) get8<T, TPR, NV, VEC>(x, d, t, k, h[k]);
  if (a.residual) {
    const T* r = reinterpret_cast<const T*>(a.residual) + row0 * a.ldr;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float v[8];
      get8<T, TPR, NV, VEC>(r, d, t, k, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = rounded<T>(h[k][e] + v[e]);
    }
  }
  if (a.H) {
    T* o = reinterpret_cast<T*>(a.H) + row0 * (int64_t)d;
#pragma unroll
    for (int k = 0; k < NV; ++k) put8<T, TPR, NV, VEC>(o, d, t, k, h[k]);
  }
  double s = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)h[k][e], (double)h[k][e], s);
  s = row_join64<TPR>(s, red64) * (1.0 / d) + (double)a.eps;
  const double r64 = rsqrt64(s);
  const float rstd = (float)r64;
  if (a.rstd && t == 0) a.rstd[row0] = rstd;
  const T* w = reinterpret_cast<const T*>(a.weight);
  float y[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    float v[8];
    get8<T, TPR, NV, VEC>(w, d, t, k, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[k][e] = h[k][e] * rstd * v[e];
  }
  if (a.Y) {
    T* o = reinterpret_cast<T*>(a.Y) + row0 * (int64_t)d;
#pragma unroll
    for (int k = 0; k < NV; ++k) put8<T, TPR, NV, VEC>(o, d, t, k, y[k]);
  }
  if constexpr (PACK) {
    pack_row<TPR, NV, VEC, true>(y, d, t, a.codes + row0 * (int64_t)d, a.scale8 + row0, red, [&](int k, double (&v)[8]) {
      float f[8];
      get8<T, TPR, NV, VEC>(w, d, t, k, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = h[0][e];
#pragma unroll
        for (int i = 1; i < NV; ++i) x = k == i ? h[i][e] : x;
        v[e] = (double)x * r64 * (double)f[e];
      }
    });
  }
}

// Any activation's rows in 8 bits: a stream (8192 x 14336 bf16: 352 MB in 55 to 62 us,
// 6 TB/s).  No border cases: the values are what is rounded.
template <typename T, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__((Row<TPR, NV, VEC>::NT)) act8_pack_kernel(const T* X, int64_t ldx, int64_t M, int d,
                                                                            uint8_t* codes, float* scale8) {
  using R = Row<TPR, NV, VEC>;
  __shared__ float red[16];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * R::RPB + threadIdx.x / TPR;
  if (TPR < 256 && row >= M) return;
  float x[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) get8<T, TPR, NV, VEC>(X + row * ldx, d, t, k, x[k]);
  pack_row<TPR, NV, VEC, false>(x, d, t, codes + row * (int64_t)d, scale8 + row, red, [](int, double (&)[8]) {});
}

// x = code * scale in the type: 8 elements a thread.
__device__ __forceinline__ void decode4(uint32_t v, float s, float* f) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
  f[0] = lo[0] * s;
  f[1] = lo[1] * s;
  f[2] = hi[0] * s;
  f[3] = hi[1] * s;
}
template <typename T>
__global__ void __launch_bounds__(256) act8_unpack_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scale8,
                                                          int64_t M, int64_t d, T* __restrict__ X) {
  const int64_t n = M * d, per = (int64_t)gridDim.x * 256 * 8;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += per) {
    if (d % 8 == 0) {  // (a chunk lies in one row)
      const u32x2 v = *reinterpret_cast<const u32x2*>(codes + i);
      const float s = scale8[i / d];
      float f[8];
      decode4(v[0], s, f);
      decode4(v[1], s, f + 4);
      if constexpr (sizeof(T) == 2) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
        *reinterpret_cast<u32x4*>(X + i) = o;
      } else {
        *reinterpret_cast<f32x4*>(X + i) = f32x4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4*>(X + i + 4) = f32x4{f[4], f[5], f[6], f[7]};
      }
    } else {
      for (int64_t j = i; j < min(i + 8, n); ++j) {
        float f[4];
        decode4(codes[j], scale8[j / d], f);
        store_out<T>(X, j, f[0]);
      }
    }
  }
}

// Two arrays of gradients to bf16, for backwards that form them in fp32.
__global__ void __launch_bounds__(256) to_bf16_kernel(const float* a, int64_t na, uint16_t* oa, const float* b, int64_t nb, uint16_t* ob) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < na + nb; i += (int64_t)gridDim.x * 256)
    if (i < na)
      oa[i] = f2bf(a[i]);
    else
      ob[i - na] = f2bf(b[i - na]);
}

// ---------------------------------------------------------------------------
// backward: with xh = h rstd and g = dY w,
//     dX = rstd (g - xh mean(g xh)) + dH,   dw = sum over rows of dY xh
// Blocks take rows in turn; a thread keeps its columns' sums of dw in
// registers, the block's are joined in LDS and left in part [blocks, d], which
// rmsnorm_dw_kernel sums in order.  Up to 1024 blocks, four a CU: enough loads in
// flight for the memory's rate (8192 x 4096 bf16 with dH: 268 MB in 50 us, 5.4 TB/s)
// and 16 MB of partials (4 us); 512 of rows past 8192, whose registers fill a CU with two.
// Past 16384 elements the registers do not hold a row's x, g and sums (48 to 127 of them
// spill in the row loop): 2048 x 32768 with dH 260 us, 2 TB/s; x 16384 53 us.
// ---------------------------------------------------------------------------
template <typename T, int TPR, int NV, bool VEC>
__global__ void __launch_bounds__((Row<TPR, NV, VEC>::NT)) rmsnorm_grad_kernel(const RmsNormGradArgs a) {
  using R = Row<TPR, NV, VEC>;
  __shared__ float red[16];
  __shared__ float joined[TPR < 256 ? R::NT * 8 : 1];
  const int t = threadIdx.x % TPR;
  const int d = a.d;
  float dw[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = 0.f;
  const T* w = reinterpret_cast<const T*>(a.weight);
  for (int64_t row = (int64_t)blockIdx.x * R::RPB + threadIdx.x / TPR; row < a.M; row += (int64_t)gridDim.x * R::RPB) {
    const int64_t o = row * (int64_t)d;
    const float rstd = a.rstd[row];
    float x[NV][8], g[NV][8];
    float c = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float v[8];
      get8<T, TPR, NV, VEC>(reinterpret_cast<const T*>(a.H) + o, d, t, k, x[k]);
      get8<T, TPR, NV, VEC>(reinterpret_cast<const T*>(a.dY) + o, d, t, k, g[k]);
      get8<T, TPR, NV, VEC>(w, d, t, k, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k][e] *= rstd;
        dw[k][e] = __builtin_fmaf(g[k][e], x[k][e], dw[k][e]);
        g[k][e] *= v[e];
        c = __builtin_fmaf(g[k][e], x[k][e], c);
      }
    }
    c = row_join<TPR, false>(c, red) / (float)d;
    if (!a.dX) continue;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dH) get8<T, TPR, NV, VEC>(reinterpret_cast<const T*>(a.dH) + o, d, t, k, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(rstd, g[k][e] - x[k][e] * c, v[e]);
      put8<T, TPR, NV, VEC>(reinterpret_cast<T*>(a.dX) + o, d, t, k, v);
    }
  }
  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * d;
  if constexpr (TPR >= 256) {
#pragma unroll
    for (int k = 0; k < NV; ++k) put8<float, TPR, NV, VEC>(part, d, t, k, dw[k]);
  } else {
    // one chunk of every thread at a time: rows of the block in order
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) joined[threadIdx.x * 8 + e] = dw[k][e];
      __syncthreads();
      for (int i = threadIdx.x; i < TPR * 8; i += R::NT) {
        float s = 0.f;
        for (int q = 0; q < R::RPB; ++q) s += joined[q * TPR * 8 + i];
        const int c = R::col(i >> 3, k, i & 7);
        if (c < d) part[c] = s;
      }
    }
  }
}

// dw[c] = the sum over blocks of part[.][c]: 32 columns a block, 32 threads a
// column take every 32nd row and meet in order.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* __restrict__ part, int blocks, int d, T* __restrict__ dw) {
  __shared__ float red[32][33];
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int c = (int)blockIdx.x * 32 + l;
  float s = 0.f;
  if (c < d)
    for (int b0 = q; b0 < blocks; b0 += 32 * 8) {  // 8 loads in flight
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = b0 + 32 * k < blocks ? part[(int64_t)(b0 + 32 * k) * d + c] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && c < d) {
    float v = red[0][l];
    for (int k = 1; k < 32; ++k) v += red[k][l];
    store_out<T>(dw, c, v);
  }
}

// f(TPR, NV) of the narrowest form that holds a row.
template <class F>
void by_width(int d, F&& f) {
  using std::integral_constant;
  auto go = [&](auto tpr, auto nv) { f(tpr, nv); };
#define FORM(T, N) go(integral_constant<int, T>{}, integral_constant<int, N>{})
  if (d <= 128)
    FORM(16, 1);
  else if (d <= 256)
    FORM(16, 2);
  else if (d <= 512)
    FORM(64, 1);
  else if (d <= 1024)
    FORM(64, 2);
  else if (d <= 2048)
    FORM(256, 1);
  else if (d <= 4096)
    FORM(256, 2);
  else if (d <= 8192)
    FORM(256, 4);
  else if (d <= 16384)
    FORM(1024, 2);
  else
    FORM(1024, 4);
#undef FORM
}

bool vec16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// f(first row, rows) of launches that take every row: a launch has fewer than 2^32
// threads, 2^24 blocks of 256.
template <class R, class F>
void by_rows(int64_t M, F&& f) {
  constexpr int64_t most = int64_t(UINT32_MAX / R::NT) * R::RPB;
  for (int64_t r0 = 0; r0 < M; r0 += most) f(r0, std::min(most, M - r0));
}
template <class R>
dim3 row_blocks(int64_t M) { return dim3((unsigned)((M + R::RPB - 1) / R::RPB)); }

template <typename T>
RmsNormArgs rows_of(RmsNormArgs a, int64_t r0, int64_t rows) {
  auto in = [&](const void*& p, int64_t ld) { p = p ? static_cast<const T*>(p) + r0 * ld : nullptr; };
  auto out = [&](void*& p) { p = p ? static_cast<T*>(p) + r0 * a.d : nullptr; };
  in(a.X, a.ldx);
  in(a.residual, a.ldr);
  out(a.H);
  out(a.Y);
  if (a.codes) a.codes += r0 * a.d;
  if (a.scale8) a.scale8 += r0;
  if (a.rstd) a.rstd += r0;
  a.M = rows;
  return a;
}

template <typename T, bool VEC>
void run_norm(const RmsNormArgs& all, hipStream_t st) {
  by_width(all.d, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    using R = Row<TPR, NV, VEC>;
    by_rows<R>(all.M, [&](int64_t r0, int64_t rows) {
      const RmsNormArgs a = rows_of<T>(all, r0, rows);
      if (a.codes)
        hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, NV, VEC, true>), row_blocks<R>(rows), dim3(R::NT), 0, st, a);
      else
        hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, NV, VEC, false>), row_blocks<R>(rows), dim3(R::NT), 0, st, a);
    });
  });
}

template <typename T, bool VEC>
void run_pack(const void* X, int64_t ldx, int64_t M, int d, uint8_t* codes, float* scale8, hipStream_t st) {
  by_width(d, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    using R = Row<TPR, NV, VEC>;
    by_rows<R>(M, [&](int64_t r0, int64_t rows) {
      hipLaunchKernelGGL((act8_pack_kernel<T, TPR, NV, VEC>), row_blocks<R>(rows), dim3(R::NT), 0, st,
                         static_cast<const T*>(X) + r0 * ldx, ldx, rows, d, codes + r0 * d, scale8 + r0);
    });
  });
}

template <typename T, bool VEC>
void run_grad(const RmsNormGradArgs& a, int blocks, hipStream_t st) {
  by_width(a.d, [&](auto tpr, auto nv) {
    constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
    hipLaunchKernelGGL((rmsnorm_grad_kernel<T, TPR, NV, VEC>), dim3((unsigned)blocks), dim3(Row<TPR, NV, VEC>::NT), 0, st, a);
  });
}

}  // namespace

hipError_t launch_rmsnorm(int elem_bytes, const RmsNormArgs& a, hipStream_t st) {
  if (a.M <= 0) return hipSuccess;
  if (a.d < 1 || a.d > kNormMaxDim || a.M > INT32_MAX) return hipErrorInvalidValue;
  const bool vec = a.d % 8 == 0 && a.ldx % 8 == 0 && a.ldr % 8 == 0 && vec16(a.X) && vec16(a.residual) && vec16(a.weight) &&
                   vec16(a.H) && vec16(a.Y) && (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0;
  if (elem_bytes == 2)
    vec ? run_norm<uint16_t, true>(a, st) : run_norm<uint16_t, false>(a, st);
  else
    vec ? run_norm<float, true>(a, st) : run_norm<float, false>(a, st);
  return hipGetLastError();
}

hipError_t launch_act8_pack(int elem_bytes, const void* X, int64_t ldx, int64_t M, int d, uint8_t* codes, float* scale8,
                            hipStream_t st) {
  if (M <= 0) return hipSuccess;
  if (d < 1 || d > kNormMaxDim || M > INT32_MAX) return hipErrorInvalidValue;
  const bool vec = d % 8 == 0 && ldx % 8 == 0 && vec16(X) && (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  if (elem_bytes == 2)
    vec ? run_pack<uint16_t, true>(X, ldx, M, d, codes, scale8, st) : run_pack<uint16_t, false>(X, ldx, M, d, codes, scale8, st);
  else
    vec ? run_pack<float, true>(X, ldx, M, d, codes, scale8, st) : run_pack<float, false>(X, ldx, M, d, codes, scale8, st);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(int elem_bytes, const uint8_t* codes, const float* scale8, int64_t M, int64_t d, void* X,
                              hipStream_t st) {
  if (M <= 0) return hipSuccess;
  if (d < 1 || d > kNormMaxDim || M > INT32_MAX) return hipErrorInvalidValue;
  const int64_t chunks = (M * d + 7) / 8;
  const unsigned blocks = (unsigned)std::min<int64_t>((chunks + 255) / 256, 256 * 16);
  if (elem_bytes == 2)
    hipLaunchKernelGGL((act8_unpack_kernel<uint16_t>), dim3(blocks), dim3(256), 0, st, codes, scale8, M, d, static_cast<uint16_t*>(X));
  else
    hipLaunchKernelGGL((act8_unpack_kernel<float>), dim3(blocks), dim3(256), 0, st, codes, scale8, M, d, static_cast<float*>(X));
  return hipGetLastError();
}

hipError_t launch_to_bf16(const float* a, int64_t na, uint16_t* oa, const float* b, int64_t nb, uint16_t* ob, hipStream_t st) {
  const unsigned blocks = (unsigned)std::max<int64_t>(1, std::min<int64_t>((na + nb + 255) / 256, 2048));
  hipLaunchKernelGGL(to_bf16_kernel, dim3(blocks), dim3(256), 0, st, a, na, oa, b, nb, ob);
  return hipGetLastError();
}

int rmsnorm_grad_blocks(int64_t M, int d) {
  const int rows = d <= 256 ? 16 : d <= 1024 ? 4 : 1;  // of a block
  return (int)std::max<int64_t>(1, std::min<int64_t>((M + rows - 1) / rows, d > 8192 ? 512 : 1024));
}

hipError_t launch_rmsnorm_grad(int elem_bytes, const RmsNormGradArgs& a, void* dw, int dw_bytes, hipStream_t st) {
  if (a.d < 1 || a.d > kNormMaxDim || a.M > INT32_MAX || (dw && !a.part)) return hipErrorInvalidValue;
  const int blocks = rmsnorm_grad_blocks(a.M, a.d);
  const bool vec = a.d % 8 == 0 && vec16(a.H) && vec16(a.dY) && vec16(a.dH) && vec16(a.dX) && vec16(a.weight) && vec16(a.part);
  if (elem_bytes == 2)
    vec ? run_grad<uint16_t, true>(a, blocks, st) : run_grad<uint16_t, false>(a, blocks, st);
  else
    vec ? run_grad<float, true>(a, blocks, st) : run_grad<float, false>(a, blocks, st);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dw) return e;
  const dim3 grid((unsigned)((a.d + 31) / 32));
  if (dw_bytes == 2)
    hipLaunchKernelGGL((rmsnorm_dw_kernel<uint16_t>), grid, dim3(1024), 0, st, a.part, blocks, a.d, static_cast<uint16_t*>(dw));
  else
    hipLaunchKernelGGL((rmsnorm_dw_kernel<float>), grid, dim3(1024), 0, st, a.part, blocks, a.d, static_cast<float*>(dw));
  return hipGetLastError();
}

}  // namespace lora
