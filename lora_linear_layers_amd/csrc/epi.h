// epi.h - the epilogue of a LoRA linear layer beyond its product: bias,
// activation and residual,
//
//     Z = X W^T + s (X A^T) B^T + b,   Y = act(Z) + R
//
// (page "Unsloth框架：高效LLM微调与LoRA优化实践", section 3.1: the graph rewriter
// merges a linear layer with its neighbours).  Z is formed and activated in
// fp32, straight from the product's accumulators: Y is rounded once, and Z
// once more where it is kept for a backward, in the layer's type as every
// activation that a training step keeps (fp32 would double its M d_out bytes,
// written and read again): act'(Z) moves by at most 2^-8 |z| times 0.5 (SiLU) or
// 0.8 (GELU), 0.0006 of a gradient in the mean, where a gradient's own rounding
// to bf16 is 0.0017.  The epilogue reads R and writes
// Y (and Z) once, so it costs the product's kernels little: a 256 x 256 tile's
// fixed time is 15.5 us against 11 for a plain store (16 to 24 with SiLU or
// GELU, residual and Z), 8192 x 4096 over 14336 with residual runs at 1300
// TFLOP/s, and the few-token kernels' times are the plain layer's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_SILU = 2, ACT_GELU = 3, ACT_GELU_TANH = 4 };

// bias [N], res [M, N] and z [M, N] in the layer's type, rows as long as the
// output's; a NULL one is absent.  res may be the output itself: the thread
// that stores an element is the one that read it.
struct EpiArgs {
  const void* bias;
  const void* res;
  void* z;
  int act;
};

// Rows with an adapter of their own, added where a product of few rows is
// finished: y[t, c] += P[t, :] . B[a][c, :], a = index[t] (none outside [0, n)),
// P fp32 [M, r], B bf16 [n][N, r], r a multiple of 8.
struct StripArgs {
  const float* P;
  const int* index;
  const uint16_t* B;
  int n, r;
};

// P(N(0, 1) > a) for a >= 0: e^(-a^2/2) t q(t), t = 1 / (1 + 0.32 a), q fitted
// to the scaled complementary error function (relative error below 1.7e-5,
// far below half a bf16 step).  gelu(z) = z P(N < z) keeps its relative
// accuracy in the negative tail this way; 1 - erf would lose it.
__device__ __forceinline__ float normal_tail_fast(float a) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.32f, a, 1.f));
  float q = -0.06501922f;
  q = __builtin_fmaf(q, t, 0.13521868f);
  q = __builtin_fmaf(q, t, 0.05355598f);
  q = __builtin_fmaf(q, t, 0.12148202f);
  q = __builtin_fmaf(q, t, 0.12709288f);
  q = __builtin_fmaf(q, t, 0.12767541f);
  return __expf(-0.5f * a * a) * t * q;
}

// P(N(0, 1) <= z)
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z) {
  if constexpr (FAST) {
    const float t = normal_tail_fast(fabsf(z));
    return z < 0.f ? t : 1.f - t;
  } else {
    return 0.5f * erfcf(-0.70710678118654752f * z);
  }
}

template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (FAST)
    return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  else
    return 1.f / (1.f + expf(-z));
}

// sqrt(2 / pi) (z + 0.044715 z^3); tanh(u) = 2 sigmoid(2 u) - 1, so
// gelu_tanh(z) = z sigmoid(2 u)
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  return 0.79788456080286536f * __builtin_fmaf(0.044715f * z * z, z, z);
}

// FAST: outputs in bf16 (hardware exponential and reciprocal, about 1e-6
// relative); else fp32.
template <bool FAST>
__device__ __forceinline__ float act_fwd(float z, int act) {
  switch (act) {
    case ACT_RELU: return z < 0.f ? 0.f : z;  // (a NaN stays)
    case ACT_SILU: return z * sigmoid<FAST>(z);
    case ACT_GELU: return z * normal_cdf<FAST>(z);
    case ACT_GELU_TANH: return z * sigmoid<FAST>(2.f * gelu_tanh_arg(z));
    default: return z;
  }
}

template <bool FAST>
__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case ACT_SILU: {
      const float s = sigmoid<FAST>(z);
      return s * (1.f + z * (1.f - s));
    }
    case ACT_GELU: {
      const float phi = 0.39894228040143268f * (FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z));
      return normal_cdf<FAST>(z) + z * phi;
    }
    case ACT_GELU_TANH: {
      const float s = sigmoid<FAST>(2.f * gelu_tanh_arg(z));
      const float w = s * (1.f - s);  // (0 far out, where z^2 may be infinite)
      return w == 0.f ? s : s + 2.f * z * w * 0.79788456080286536f * (1.f + 3.f * 0.044715f * z * z);
    }
    default: return 1.f;
  }
}

// act over a few values at once: one uniform branch for all of them
template <bool FAST, int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = act_fwd<FAST>(v[e], ACT_RELU);
      break;
    case ACT_SILU:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = act_fwd<FAST>(v[e], ACT_SILU);
      break;
    case ACT_GELU:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = act_fwd<FAST>(v[e], ACT_GELU);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = act_fwd<FAST>(v[e], ACT_GELU_TANH);
      break;
    default: break;
  }
}

// g *= act'(z); what relu stops stays out whatever it is (an infinity times 0 is
// no gradient)
template <bool FAST, int N>
__device__ __forceinline__ void act_grad_all(float (&g)[N], const float (&z)[N], int act) {
  switch (act) {
    case ACT_RELU:
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] = z[e] > 0.f ? g[e] : 0.f;
      break;
    case ACT_SILU:
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] *= act_grad<FAST>(z[e], ACT_SILU);
      break;
    case ACT_GELU:
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] *= act_grad<FAST>(z[e], ACT_GELU);
      break;
    case ACT_GELU_TANH:
#pragma unroll
      for (int e = 0; e < N; ++e) g[e] *= act_grad<FAST>(z[e], ACT_GELU_TANH);
      break;
    default: break;
  }
}

// N consecutive elements (N = 4 or 8) of a T array (bf16 patterns or fp32) at
// an address aligned to N elements (16 bytes where that is less) as floats,
// and back
template <int N>
__device__ __forceinline__ void epi_load(const uint16_t* p, float (&f)[N]) {
  typedef uint32_t V __attribute__((ext_vector_type(N / 2)));
  const V v = *reinterpret_cast<const V*>(p);
#pragma unroll
  for (int k = 0; k < N / 2; ++k) {
    f[2 * k] = __builtin_bit_cast(float, v[k] << 16);
    f[2 * k + 1] = __builtin_bit_cast(float, v[k] & 0xFFFF0000u);
  }
}
template <int N>
__device__ __forceinline__ void epi_load(const float* p, float (&f)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + k);
    f[k] = v.x;
    f[k + 1] = v.y;
    f[k + 2] = v.z;
    f[k + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void epi_store(uint16_t* p, const float (&f)[N]) {
  typedef uint32_t V __attribute__((ext_vector_type(N / 2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  V v;
#pragma unroll
  for (int k = 0; k < N / 2; ++k)
    v[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{f[2 * k], f[2 * k + 1]}, b2));
  *reinterpret_cast<V*>(p) = v;
}
template <int N>
__device__ __forceinline__ void epi_store(float* p, const float (&f)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
}

// The epilogue of N consecutive columns: v holds the product; col the first
// column, o the element's offset in Y, R and Z.
template <typename T, int N>
__device__ __forceinline__ void epi_apply(const EpiArgs& ep, T* y, int64_t o, int64_t col, float (&v)[N]) {
  constexpr bool FAST = sizeof(T) == 2;
  float t[N];
  if (ep.bias) {
    epi_load(static_cast<const T*>(ep.bias) + col, t);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += t[e];
  }
  if (ep.res) epi_load(static_cast<const T*>(ep.res) + o, t);
  if (ep.z) epi_store(static_cast<T*>(ep.z) + o, v);
  act_all<FAST>(v, ep.act);
  if (ep.res) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += t[e];
  }
  epi_store(y + o, v);
}

// one element
template <typename T>
__device__ __forceinline__ float epi_ld1(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(float, (uint32_t)*p << 16);
  else
    return *p;
}
template <typename T>
__device__ __forceinline__ void epi_st1(T* p, float v) {
  if constexpr (sizeof(T) == 2)
    *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else
    *p = v;
}
template <typename T>
__device__ __forceinline__ void epi_apply1(const EpiArgs& ep, T* y, int64_t o, int64_t col, float v) {
  if (ep.bias) v += epi_ld1(static_cast<const T*>(ep.bias) + col);
  const float r = ep.res ? epi_ld1(static_cast<const T*>(ep.res) + o) : 0.f;
  if (ep.z) epi_st1(static_cast<T*>(ep.z) + o, v);
  v = act_fwd<sizeof(T) == 2>(v, ep.act);
  epi_st1(y + o, ep.res ? v + r : v);
}

}  // namespace lora
