// strip.h - rows with an adapter of their own (StripArgs, epi.h), added to the
// outputs of a product of up to 64 rows where it finishes them.
#pragma once

#include "gemm.h"

namespace lora {

// This lane's row's adapter, of the 16 rows from row0 (row lane % 16; -1: none).
__device__ __forceinline__ int strip_row(const StripArgs& s, int M, int row0) {
  const int row = row0 + (threadIdx.x & 15);
  const int a = row < M ? s.index[row] : -1;
  return a >= 0 && a < s.n ? a : -1;
}

// y[j][v] += the strips' part of row row0 + 4 (lane / 16) + v, column col[j] (of lane
// % 16), for the 16 rows from row0, adapter by adapter of theirs: a product of
// all 16 strips (in two bf16 parts, so that they keep 16 bits) with the adapter's
// columns on the matrix cores, of which its own rows are taken: nothing of another's
// reaches them, infinities and NaNs included.  The operand's 16 columns are read 64
// bytes (32 ranks) each at a time; F such loads and the next F are in flight.
// (By dot products, a lane a column, each 16 bytes of a lane came from another line: 32
// rows of rank 64, 4096 -> 4096, 61 us a call against 29, 64 rows -> 14336 107 against
// 58; at rank 16 two steps of them were 1 to 3 us shorter, 37 against 38 and 45 against 47.)
// mine: strip_row's.  Of the rows' adapters this wave takes every `parts`-th, from the `part`-th on.
template <int NJ, int F>
__device__ __forceinline__ void strip_add(const StripArgs& s, int M, int64_t N, int row0, int mine, const int64_t (&col)[NJ],
                                          float (&y)[NJ][4], int part = 0, int parts = 1) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4)));
  typedef float f4 __attribute__((ext_vector_type(4)));
  constexpr int G = NJ >= F ? 1 : F / NJ;  // adapters at a time
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int row = row0 + l16 < M ? row0 + l16 : -1;
  uint64_t left = __ballot(mine >= 0);  // rows whose adapters are still to come
  auto next = [&] {
    const int e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == e);
    return e;
  };
  auto skip = [&](int k) {
    for (; k > 0 && left; --k) next();
  };
  skip(part);
  if (!left) return;
  int own[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) own[v] = __shfl(mine, 4 * g + v);
  const float* p = s.P + (int64_t)(row >= 0 ? row : 0) * s.r;

  struct Step {
    int e[G], q0;  // adapters (-2: none), ranks from q0
    v4 w[G][NJ];
    f4 x[2];
  };
  auto load = [&](Step& t) {
    const int q = t.q0 + 8 * g;
    const bool in = row >= 0 && q < s.r;
#pragma unroll
    for (int h = 0; h < 2; ++h) t.x[h] = in ? *reinterpret_cast<const f4*>(p + q + 4 * h) : f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        t.w[k][j] = t.e[k] >= 0 && q < s.r && col[j] < N
                        ? *reinterpret_cast<const v4*>(s.B + ((int64_t)t.e[k] * N + col[j]) * s.r + q)
                        : v4{0u, 0u, 0u, 0u};
  };
  auto take = [&](Step& t) {  // the next adapters
    t.q0 = 0;
#pragma unroll
    for (int k = 0; k < G; ++k) {
      t.e[k] = -2;
      if (left) {
        t.e[k] = next();
        skip(parts - 1);
      }
    }
  };
  f4 d[G][NJ];
#pragma unroll
  for (int k = 0; k < G; ++k)
#pragma unroll
    for (int j = 0; j < NJ; ++j) d[k][j] = f4{0.f, 0.f, 0.f, 0.f};
  // computes t while n is loaded; false: t was the last
  auto step = [&](Step& t, Step& n) {
    const bool last = t.q0 + 32 >= s.r, more = !last || left;
    if (more) {
      if (last) {
        take(n);
      } else {
        n.q0 = t.q0 + 32;
#pragma unroll
        for (int k = 0; k < G; ++k) n.e[k] = t.e[k];
      }
      load(n);
    }
    v4 hi, lo;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float a = t.x[h >> 1][2 * (h & 1)], b = t.x[h >> 1][2 * (h & 1) + 1];
      const uint32_t u = pack_bf16x2(a, b);
      hi[h] = u;
      lo[h] = pack_bf16x2(a - __builtin_bit_cast(float, u << 16), b - __builtin_bit_cast(float, u & 0xFFFF0000u));
    }
#pragma unroll
    for (int k = 0; k < G; ++k)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const bf16x8 b = __builtin_bit_cast(bf16x8, t.w[k][j]);
        d[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hi), b, d[k][j], 0, 0, 0);
        d[k][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lo), b, d[k][j], 0, 0, 0);
      }
    if (last) {
#pragma unroll
      for (int k = 0; k < G; ++k)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float x = d[k][j][v];
            y[j][v] += own[v] == t.e[k] ? x : 0.f;
            d[k][j][v] = 0.f;
          }
    }
    return more;
  };
  Step a, b;
  take(a);
  load(a);
  while (step(a, b) && step(b, a)) {
  }
}

}  // namespace lora
