// loss.hip - what a LoRA training step computes behind its head projection:
// the log-probabilities of tokens from their logits, the preference loss of
// response pairs and the clipped policy loss with a KL term, each with its
// gradient, plus their host-side launchers (internal interface in launch.h).
//
// All of them are streams: a few operations per byte, so each reads its
// inputs once per direction and what bounds it is the memory's rate, or, at a
// few thousand tokens, the launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"

namespace lora {

namespace {

constexpr float LOG2E = 1.44269504088896340736f;

// 16 bytes of a row at a multiple of 4 bytes: one global_load_dwordx4, as fast
// as at a multiple of 16.  Rows of an odd bf16 vocabulary start 2 bytes off
// every other time, which costs 20 % (8192 x 127999: 427 against 349 us), so
// their first element is taken apart (row_head).
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename T>
__device__ __forceinline__ int row_head(const T* p) {
  return sizeof(T) == 2 ? (int)((reinterpret_cast<uintptr_t>(p) >> 1) & 1) : 0;
}

template <typename T>
struct Row;
template <>
struct Row<uint16_t> {  // bf16 bit patterns
  static constexpr int E = 8;
  typedef u32x4_e2 V;
  static __device__ __forceinline__ float at(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }
  static __device__ __forceinline__ u32x4 none() { return u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u}; }  // -inf
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __builtin_bit_cast(float, v[k] << 16);
      f[2 * k + 1] = __builtin_bit_cast(float, v[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pack_bf16x2(f[2 * k], f[2 * k + 1]);
    return v;
  }
};
template <>
struct Row<float> {
  static constexpr int E = 4;
  typedef u32x4_e4 V;
  static __device__ __forceinline__ float at(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  static __device__ __forceinline__ u32x4 none() { return u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}; }
  static __device__ __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u = v[k];
      f[k] = __builtin_bit_cast(float, u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    u32x4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __builtin_bit_cast(uint32_t, f[k]);
    return v;
  }
};

// ---------------------------------------------------------------------------
// log-probabilities: one pass over a row with the running maximum m and the
// rest r of the sum, that of e^(tau (z - m)) but for one element of the maximum:
// logp = tau (z_t - m) - log(1 + r).  m, and log(1 + r) from r alone, are kept
// apart (the log-sum-exp, or 1 + r, would round away what a confident row's small
// log-probability is made of).
// Bound by reading the logits and, not far behind, by the instructions: 8192 x
// 128000 bf16 in 333 us, 6.3 TB/s (a large copy moves 5.2 TB/s, read and
// written; with the sum in one number and its digits lost, 328 us); the
// exponential, a quarter-rate instruction, would take 0.11 ms of it.  More than 64
// registers a thread would leave one block of 1024 a CU (432 us).  The gradient
// reads and writes them once: 671 us behind the forward, 6.2 TB/s.  24 x 32000:
// 6.6 us, a launch, one round of loads and the joins.  (Medians of calls 100 to
// 200 of a loop.)
// ---------------------------------------------------------------------------
__device__ __forceinline__ float fexp2(float x) { return __builtin_amdgcn_exp2f(x); }

// A part of a row is (m, r): its maximum and the sum of e^(tau (z - m)) over its
// other elements, one element of the maximum left out, so that the sum is 1 + r.
// Held in one number, 1 + r would round away the digits of a small r, which are
// all that a confident row's log-probability -log(1 + r) is made of.  A part
// with no finite value has m = -inf, r = 0 and adds nothing.  c = tau log2 e.
__device__ __forceinline__ void join_max_rest(float& m, float& r, float m2, float r2, float c) {
  const float nm = fmaxf(m, m2), base = nm == -INFINITY ? 0.f : nm;
  const float f = fexp2((m - base) * c), f2 = fexp2((m2 - base) * c);
  r = r * f + r2 * f2 + fminf(f, f2);  // (the lower maximum joins the rest)
  m = nm;
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8, 8))) token_logp_kernel(const T* __restrict__ z, int64_t ld, int64_t rows, int V,
                                                        const int64_t* __restrict__ target, float tau,
                                                        float* __restrict__ logp, float* __restrict__ stats) {
  using R = Row<T>;
  constexpr int E = R::E, U = 4, G = 2;
  __shared__ float red[2][NT / 64];
  const float c = tau * LOG2E;
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* zr = z + row * ld;
    const int64_t t = target[row];
    const bool has = t >= 0 && t < V;
    const float zt = has ? R::at(zr + t) : 0.f;
    // top: the vector that brought the thread's maximum, st: its sum with the
    // maximum in it, sr: the sum of all the other vectors
    float m = -INFINITY, st = 0.f, sr = 0.f;
    u32x4 top = {0u, 0u, 0u, 0u};
    auto take = [&](const u32x4* v) {  // G vectors at one scale: one rescaling for all of them
      float cm[G], nm = m;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        float x[E];
        R::unpack(v[u], x);
        cm[u] = x[0];
#pragma unroll
        for (int e = 1; e < E; ++e) cm[u] = fmaxf(cm[u], x[e]);
        nm = fmaxf(nm, cm[u]);
      }
      const float base = nm == -INFINITY ? 0.f : nm, f = fexp2((m - base) * c);
      sr *= f;
      st *= f;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        float x[E], sv = 0.f;
        R::unpack(v[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) sv += fexp2((x[e] - base) * c);
        const bool up = cm[u] > m;
        sr += up ? st : sv;
        st = up ? sv : st;
#pragma unroll
        for (int k = 0; k < 4; ++k) top[k] = up ? v[u][k] : top[k];
        m = up ? cm[u] : m;
      }
    };
    const int head = row_head(zr), nv = (V - head) / E;
    const T* zv = zr + head;
    auto vec = [&](int k) { return *reinterpret_cast<const typename R::V*>(zv + (int64_t)k * E); };
    int i = tid;
    u32x4 v[U];
    for (; i + (U - 1) * NT < nv; i += U * NT) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = vec(i + u * NT);
#pragma unroll
      for (int u = 0; u < U; u += G) take(v + u);
    }
    if (i < nv) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = R::none();
        if (i + u * NT < nv) v[u] = vec(i + u * NT);
      }
#pragma unroll
      for (int u = 0; u < U; u += G) take(v + u);
    }
    float r = sr;
    if (m > -INFINITY) {  // the rest of the top vector, one element of the maximum left out
      float x[E];
      R::unpack(top, x);
      bool left = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool here = !left && x[e] == m;
        r += here ? 0.f : fexp2((x[e] - m) * c);
        left = left || here;
      }
    }
    // the elements before and behind the vectors (at most E)
    const int rest = V - head - nv * E;
    if (tid < rest + head) join_max_rest(m, r, tid < rest ? R::at(zv + (int64_t)nv * E + tid) : R::at(zr), 0.f, c);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float m2 = __shfl_xor(m, o), r2 = __shfl_xor(r, o);
      join_max_rest(m, r, m2, r2, c);
    }
    if constexpr (NT > 64) {
      if ((tid & 63) == 0) {
        red[0][tid >> 6] = m;
        red[1][tid >> 6] = r;
      }
      __syncthreads();
      if (tid < 64) {  // (the first wave alone: by every thread it would be a fifth of the row's instructions)
        m = tid < NT / 64 ? red[0][tid] : -INFINITY;
        r = tid < NT / 64 ? red[1][tid] : 0.f;
#pragma unroll
        for (int o = NT / 128; o > 0; o >>= 1) {
          const float m2 = __shfl_xor(m, o), r2 = __shfl_xor(r, o);
          join_max_rest(m, r, m2, r2, c);
        }
      }
    }
    if (tid == 0) {
      const float ls = m == -INFINITY ? logf(r) : log1pf(r);
      logp[row] = has ? (zt - m) * tau - ls : 0.f;
      stats[2 * row] = m;
      stats[2 * row + 1] = ls;
    }
    if constexpr (NT > 64) __syncthreads();  // red is free for the next row
  }
}

// dz_j = g tau (1[j = t] - e^(tau (z_j - m) - log(1 + r))).  A row without a token
// or with g = 0 is not read: its gradient is zero whatever it holds.  dz may
// be z (every thread reads its elements before it writes them).
// STREAM: past the caches (logits that exceed the 256 MB of the last level,
// which neither this pass nor the next finds there: 8192 x 128000 bf16 805 ->
// 758 us, 2047 x 50001 fp32 152 -> 140).
constexpr int GRAD_U = 4, GRAD_NT = 256;

template <typename T, bool STREAM>
__global__ void __launch_bounds__(GRAD_NT) token_logp_grad_kernel(const T* z, int64_t ld, int64_t rows, int V, int segs,
                                                                  const int64_t* __restrict__ target, float tau,
                                                                  const float* __restrict__ stats,
                                                                  const float* __restrict__ dlogp, T* dz,
                                                                  int64_t ldd) {
  using R = Row<T>;
  constexpr int E = R::E, U = GRAD_U, NT = GRAD_NT;
  const int64_t items = rows * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / segs;
    const int seg = (int)(it - row * segs);
    const int64_t t = target[row];
    const float g = t >= 0 && t < V ? dlogp[row] * tau : 0.f;
    const T* zr = z + row * ld;
    T* dr = dz + row * ldd;
    const int head = row_head(zr), nv = (V - head) / E;
    const bool zero = g == 0.f;
    const float m = stats[2 * row], ls = stats[2 * row + 1], ls2 = ls * LOG2E, c = tau * LOG2E;
    auto grad = [&](float x, int64_t j) { return (j == t ? g : 0.f) - g * fexp2((x - m) * c - ls2); };
    // the target's own: g (1 - p), from p = 1/2 on with 1 - p as -(e^logp - 1),
    // which keeps its digits where p is near 1
    auto grad_t = [&](float x) {
      const float p = fexp2((x - m) * c - ls2);
      return p < 0.5f ? g - g * p : -g * expm1f((x - m) * tau - ls);
    };
    const int i0 = seg * (U * NT) + threadIdx.x;
    u32x4 v[U];
    if (!zero) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * NT < nv) {
          const typename R::V* q = reinterpret_cast<const typename R::V*>(zr + head + (int64_t)(i0 + u * NT) * E);
          if constexpr (STREAM)
            v[u] = __builtin_nontemporal_load(q);
          else
            v[u] = *q;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = head + (int64_t)(i0 + u * NT) * E;
      if (i0 + u * NT >= nv) continue;
      u32x4 o = {0u, 0u, 0u, 0u};
      if (!zero) {
        float x[E];
        R::unpack(v[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = grad(x[e], j + e);
        o = R::pack(x);
      }
      if constexpr (STREAM)
        __builtin_nontemporal_store(o, reinterpret_cast<typename R::V*>(dr + j));
      else
        *reinterpret_cast<typename R::V*>(dr + j) = o;
    }
    // the target's element again, by the thread whose vector holds it (in place
    // of the compare above, or with the loads unconditional, the pass over 8192 x
    // 128000 takes 687 us instead of 671)
    const int vt = (int)t - head < 0 ? nv : ((int)t - head) / E, dt = vt - i0;
    if (!zero && vt < nv && dt >= 0 && dt < U * NT && dt % NT == 0) {
      u32x4 w = v[0];
#pragma unroll
      for (int u = 1; u < U; ++u) w = dt == u * NT ? v[u] : w;
      float x[E], xt = 0.f;
      R::unpack(w, x);
#pragma unroll
      for (int e = 0; e < E; ++e) xt = head + vt * E + e == (int)t ? x[e] : xt;
      R::put(dr + t, grad_t(xt));
    }
    // the elements before and behind the vectors (at most E): the last
    // segment's first threads
    const int rest = V - head - nv * E;
    if (seg == segs - 1 && (int)threadIdx.x < rest + head) {
      const int64_t j = (int)threadIdx.x < rest ? head + (int64_t)nv * E + threadIdx.x : 0;
      const float x = zero ? 0.f : R::at(zr + j);
      R::put(dr + j, zero ? 0.f : (j == t ? grad_t(x) : grad(x, j)));
    }
  }
}

template <typename T>
hipError_t run_logp(const T* z, int64_t ld, int64_t rows, int64_t V, const int64_t* target, float tau, float* logp,
                    float* stats, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(rows, 1 << 20);
  auto go = [&](auto nt_c) {
    constexpr int NT = decltype(nt_c)::value;
    hipLaunchKernelGGL((token_logp_kernel<T, NT>), dim3(grid), dim3(NT), 0, st, z, ld, rows, (int)V, target, tau, logp,
                       stats);
    return hipGetLastError();
  };
  // threads a row (measured): a wave for a short one; 1024 where the row holds
  // three rounds of their loads (8192 x 96000 bf16: 255 us against 269 with
  // 256; 8192 x 50000: 167 against 147), or the rows alone do not fill the
  // chip (64 x 128000: 13.1 us against 17.1)
  if (V <= 2048) return go(std::integral_constant<int, 64>{});
  if (V / Row<T>::E < 3 * 4 * 1024 && rows >= 512) return go(std::integral_constant<int, 256>{});
  return go(std::integral_constant<int, 1024>{});
}

template <typename T>
hipError_t run_logp_grad(const T* z, int64_t ld, int64_t rows, int64_t V, const int64_t* target, float tau,
                         const float* stats, const float* dlogp, T* dz, int64_t ldd, hipStream_t st) {
  const int64_t per = (int64_t)GRAD_U * GRAD_NT * Row<T>::E;
  const int64_t segs = std::max<int64_t>(1, (V + per - 1) / per);
  const unsigned grid = (unsigned)std::min<int64_t>(rows * segs, 1 << 22);
  if (rows * V * (int64_t)sizeof(T) > (int64_t(256) << 20))
    hipLaunchKernelGGL((token_logp_grad_kernel<T, true>), dim3(grid), dim3(GRAD_NT), 0, st, z, ld, rows, (int)V,
                       (int)segs, target, tau, stats, dlogp, dz, ldd);
  else
    hipLaunchKernelGGL((token_logp_grad_kernel<T, false>), dim3(grid), dim3(GRAD_NT), 0, st, z, ld, rows, (int)V,
                       (int)segs, target, tau, stats, dlogp, dz, ldd);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_token_logp(int elem_bytes, const void* z, int64_t ld, int64_t rows, int64_t V, const int64_t* target,
                             float tau, float* logp, float* stats, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  if (elem_bytes == 2)
    return run_logp(static_cast<const uint16_t*>(z), ld, rows, V, target, tau, logp, stats, st);
  return run_logp(static_cast<const float*>(z), ld, rows, V, target, tau, logp, stats, st);
}

hipError_t launch_token_logp_grad(int elem_bytes, const void* z, int64_t ld, int64_t rows, int64_t V,
                                  const int64_t* target, float tau, const float* stats, const float* dlogp, void* dz,
                                  int64_t ldd, hipStream_t st) {
  if (rows <= 0) return hipSuccess;
  if (elem_bytes == 2)
    return run_logp_grad(static_cast<const uint16_t*>(z), ld, rows, V, target, tau, stats, dlogp,
                         static_cast<uint16_t*>(dz), ldd, st);
  return run_logp_grad(static_cast<const float*>(z), ld, rows, V, target, tau, stats, dlogp, static_cast<float*>(dz),
                       ldd, st);
}

// ---------------------------------------------------------------------------
// The losses over packed sequences: sequence s holds the tokens [cu[s],
// cu[s + 1]) of N.  A wave takes one chunk of `ch` consecutive tokens whatever
// sequences it holds (so one long response costs no more than many short
// ones) and leaves
//   seqp[s]: the part of sequence s in the chunk it starts in,
//   head[c]: the part in chunk c of a sequence that started before it;
// a sequence's sum is seqp[s] plus head[c] over the later chunks it reaches,
// always in that order.  Sums are held in 64 bits: a preference margin is the
// difference of two sums over thousands of tokens.
// What bounds it below a million tokens is not the 17 to 21 bytes a token but
// the chain of dependent loads, so a chunk requests its tokens' values, the
// offsets of 64 sequences and what those sequences carry (advantage, weight,
// coefficient) at once, and picks the sequence's value from a lane afterwards.
// Measured on MI355X: 1.31 M tokens in 1024 sequences (27 MB), policy sums 9.5 us,
// finish 10.8, gradient 8.2; 1250 tokens in 8, the whole forward 7.0 us and the
// gradient 4.7; with a load chain per token (mask, then values) and sums through
// the LDS crossbar these were 15.6, 8.1, 14.9 and 13.3, 6.7.
// cu is read on the device and cannot be checked before the launch: every
// index that comes from it is clipped to [0, N], and tokens outside
// [cu[0], cu[S]) belong to no sequence.
// ---------------------------------------------------------------------------
namespace {

__device__ __forceinline__ int64_t clip_tok(int64_t t, int64_t N) { return t < 0 ? 0 : (t > N ? N : t); }

// lane l's value, l uniform
__device__ __forceinline__ int pick(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ float pick(float v, int l) {
  return __builtin_bit_cast(float, pick(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ int64_t pick(int64_t v, int l) {
  const uint32_t lo = (uint32_t)pick((int)(uint32_t)v, l), hi = (uint32_t)pick((int)(uint32_t)((uint64_t)v >> 32), l);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The number of sequences that end at or before token t (the first that ends
// after it), by the whole wave: a 64-way search.
__device__ __forceinline__ int first_seq(const int64_t* cu, int S, int64_t t, int lane) {
  int lo = 0, hi = S;
  while (hi > lo) {
    const int step = (hi - lo + 63) >> 6;
    const int64_t i = (int64_t)lo + (int64_t)lane * step + step - 1;
    const bool before = i < hi && cu[i + 1] <= t;
    lo += (int)__popcll(__ballot(before)) * step;
    if (step == 1) break;
    hi = min(lo + step, hi);
  }
  return min(lo, S);
}

// Walks the sequences of a stretch of tokens, by the whole wave: lane l holds
// the end of sequence base + l and that sequence's payload.
template <class Pay>
struct Walk {
  const int64_t* cu;
  int S, lane, base;
  int64_t N, end, beg0;
  const float* src[Pay::NP];  // payload arrays [S] (NULL: zeros)
  float pay[Pay::NP];

  __device__ __forceinline__ void window() {
    const int s = base + lane;
    const bool in = s < S;
    end = in ? clip_tok(cu[s + 1], N) : 0;  // (0: never past a position)
    beg0 = base < S ? clip_tok(cu[base], N) : 0;
#pragma unroll
    for (int k = 0; k < Pay::NP; ++k) pay[k] = in && src[k] ? src[k][s] : 0.f;
  }
  __device__ __forceinline__ void start(int64_t t) {
    base = S <= 64 ? 0 : first_seq(cu, S, t, lane);
    window();
  }
  // The stretch [pos, to) of [pos, t1) that lies in one sequence: its index
  // (its first token b, its lane l of the window), or -1 between sequences.
  __device__ __forceinline__ int next(int64_t pos, int64_t t1, int64_t& to, int64_t& b, int& l) {
    while (base < S) {
      const unsigned long long todo = __ballot(end > pos);
      if (todo) {
        l = __ffsll(todo) - 1;
        b = l > 0 ? pick(end, l - 1) : pick(beg0, 0);
        const int64_t e = pick(end, l);
        const int64_t stop = b > pos ? b : e;
        to = stop < t1 ? stop : t1;
        return b > pos ? -1 : base + l;
      }
      base += 64;
      if (base < S) window();
    }
    to = t1;
    return -1;
  }
};

__device__ __forceinline__ double pick(double v, int l) {
  return __builtin_bit_cast(double, pick(__builtin_bit_cast(int64_t, v), l));
}

// v + the value CTRL moves here (0 where it moves none), CTRL a data-parallel
// primitive: no trip through the LDS crossbar
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The sum over the wave, to every lane: within rows of 16 lanes (shifts by
// 1, 2, 4, 8), then lane 15 of rows 0 and 2 into rows 1 and 3, then lane 31
// into rows 2 and 3; lane 63 has it all.
__device__ __forceinline__ double wave_sum(double v) {
  v = dpp_add<0x111, 0xf>(v);
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);
  v = dpp_add<0x143, 0xc>(v);
  return pick(v, 63);
}
__device__ __forceinline__ int count(bool b) { return (int)__popcll(__ballot(b)); }

// Tokens of a wave's step: 64 lanes x UT, all their loads in flight at once.
constexpr int UT = 4, STEP = 64 * UT;

// A term adds a token's values to ND sums of its lane and counts NC properties
// over the wave; in: the token counts, in the stretch at hand.
// preference: the log-ratios and the number of counted tokens
struct PrefTerm {
  static constexpr int ND = 1, NC = 1, NV = ND + NC;
  struct Pay {
    static constexpr int NP = 1;
  };
  struct Raw {
    float lp, ref;
  };
  const float* logp;
  const float* ref;
  __device__ __forceinline__ void payload(const float* (&src)[1]) const { src[0] = nullptr; }
  __device__ __forceinline__ Raw load(int64_t t) const { return Raw{logp[t], ref ? ref[t] : 0.f}; }
  __device__ __forceinline__ void add(const Raw& r, bool in, const float (&)[1], double (&v)[ND], int (&n)[NC]) const {
    v[0] += in ? (double)r.lp - (double)r.ref : 0.0;
    n[0] += count(in);
  }
};

// e^x for a log-ratio x: the hardware's base-2 exponential of the rounded
// product.  Relative error of a normal result: (2 + 1.25 |x|) 2^-24, of which the
// exponential is 2, the product's rounding |x| and fp32's log2 e (off by 0.22 of
// its 2^-24) the rest; below 2^-126 the result is 0
__device__ __forceinline__ float exp_ratio(float x) { return fexp2(x * LOG2E); }

// e^d - d - 1: its series where the three cancel (cut after d^9: the rest is
// below 2.5e-9 of the sum, at d = -0.5).  Next to the switch at 0.5 the difference
// of the three is off by up to 35 2^-24 of itself: e^d carries most of that
__device__ __forceinline__ float kl_term(float d) {
  float q = 1.f / 362880;
  q = __builtin_fmaf(q, d, 1.f / 40320);
  q = __builtin_fmaf(q, d, 1.f / 5040);
  q = __builtin_fmaf(q, d, 1.f / 720);
  q = __builtin_fmaf(q, d, 1.f / 120);
  q = __builtin_fmaf(q, d, 1.f / 24);
  q = __builtin_fmaf(q, d, 1.f / 6);
  q = __builtin_fmaf(q, d, 0.5f);
  return fabsf(d) < 0.5f ? d * d * q : exp_ratio(d) - 1.f - d;
}

// e^d - 1: d and the sum's own series where the two cancel
__device__ __forceinline__ float kl_slope(float d) {
  return fabsf(d) < 0.5f ? d + kl_term(d) : exp_ratio(d) - 1.f;
}

struct PolicyArgs {
  const float* logp;
  const float* old;
  const float* ref;
  const float* adv;
  int adv_per_token;
  double log_lo, log_hi;  // the clip borders of logp - old: log(1 - eps_low), log(1 + eps_high)
  float r_lo, r_hi;       // and of the ratio itself
  float beta;
  struct Raw {
    float lp, old, ref, adv;
  };
  __device__ __forceinline__ Raw load(int64_t t) const {
    Raw r;
    r.lp = logp[t];
    r.old = old ? old[t] : r.lp;
    r.ref = ref ? ref[t] : r.lp;
    r.adv = adv_per_token ? adv[t] : 0.f;
    return r;
  }
};

// The clip borders are compared on logp - old in 64 bits, where the difference
// of two fp32 values is exact: a ratio rounded to fp32 first could fall on the
// other side of its border.
struct PolicyTok {
  float ratio, adv;
  bool cut;  // the clipped branch holds: no gradient through the ratio
};
__device__ __forceinline__ PolicyTok policy_tok(const PolicyArgs& p, const PolicyArgs::Raw& r, float seq_adv) {
  PolicyTok k;
  k.adv = p.adv_per_token ? r.adv : seq_adv;
  const double d = p.old ? (double)r.lp - (double)r.old : 0.0;
  const bool over = k.adv > 0.f && d > p.log_hi, under = k.adv < 0.f && d < p.log_lo;
  k.cut = over || under;
  k.ratio = over ? p.r_hi : (under ? p.r_lo : exp_ratio((float)d));
  return k;
}

struct PolicyTerm {
  static constexpr int ND = 2, NC = 2, NV = ND + NC;
  struct Pay {
    static constexpr int NP = 1;
  };
  using Raw = PolicyArgs::Raw;
  PolicyArgs p;
  __device__ __forceinline__ void payload(const float* (&src)[1]) const { src[0] = p.adv_per_token ? nullptr : p.adv; }
  __device__ __forceinline__ Raw load(int64_t t) const { return p.load(t); }
  __device__ __forceinline__ void add(const Raw& r, bool in, const float (&pay)[1], double (&v)[ND],
                                      int (&n)[NC]) const {
    const PolicyTok k = policy_tok(p, r, pay[0]);
    v[0] -= in && k.adv != 0.f ? (double)(k.ratio * k.adv) : 0.0;
    if (p.ref) v[1] += in ? (double)kl_term((float)((double)r.ref - (double)r.lp)) : 0.0;
    n[0] += count(in && k.cut);
    n[1] += count(in);
  }
};

struct SeqArgs {
  const int64_t* cu;
  const uint8_t* mask;
  int64_t N;
  int S, lg;  // a chunk: 2^lg tokens
  int64_t chunks;
  double* head;  // [chunks][NV]
  double* seqp;  // [S][NV]; then the sequences' sums
};

template <class Term>
__device__ __forceinline__ void sum_chunk(const SeqArgs& a, const Term& term, int64_t c, int lane, double* head,
                                          double* seqp) {
  constexpr int ND = Term::ND, NC = Term::NC, NV = Term::NV;
  const int64_t t0 = c << a.lg, t1 = min(t0 + (int64_t(1) << a.lg), a.N);
  Walk<typename Term::Pay> w;
  w.cu = a.cu;
  w.S = a.S;
  w.N = a.N;
  w.lane = lane;
  term.payload(w.src);
  typename Term::Raw raw[UT];
  bool keep[UT];
  auto request = [&](int64_t p) {
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      const int64_t t = p + 64 * u + lane;
      const int64_t at = t < t1 ? t : t1 - 1;  // (every lane loads, none past the chunk)
      raw[u] = term.load(at);
      keep[u] = t < t1 && (!a.mask || a.mask[at]);
    }
  };
  request(t0);
  w.start(t0);
  double v[ND];
  int n[NC];
  int cur = -1;
  bool cur_head = false;
  auto clear = [&] {
#pragma unroll
    for (int q = 0; q < ND; ++q) v[q] = 0.0;
#pragma unroll
    for (int q = 0; q < NC; ++q) n[q] = 0;
  };
  auto flush = [&] {
    if (cur < 0) return;
    double* out = cur_head ? head + c * NV : seqp + (int64_t)cur * NV;
#pragma unroll
    for (int q = 0; q < ND; ++q) v[q] = wave_sum(v[q]);
    if (lane == 0) {
#pragma unroll
      for (int q = 0; q < ND; ++q) out[q] = v[q];
#pragma unroll
      for (int q = 0; q < NC; ++q) out[ND + q] = (double)n[q];
    }
  };
  clear();
  for (int64_t p = t0; p < t1; p += STEP) {
    if (p > t0) request(p);
    const int64_t pe = min(p + STEP, t1);
    for (int64_t pos = p; pos < pe;) {
      int64_t to, b;
      int l;
      const int s = w.next(pos, pe, to, b, l);
      if (s >= 0) {
        if (s != cur) {
          flush();
          clear();
          cur = s;
          cur_head = b < t0;
        }
        float pay[1] = {pick(w.pay[0], l)};
        const int lo = (int)(pos - p), hi = (int)(to - p);
#pragma unroll
        for (int u = 0; u < UT; ++u)
          if (64 * u < hi && 64 * u + 64 > lo)  // (uniform)
            term.add(raw[u], keep[u] && 64 * u + lane >= lo && 64 * u + lane < hi, pay, v, n);
      }
      pos = to;
    }
  }
  flush();
}

// tot[s] = the sum of sequence s, for every s (one block): a lane takes a
// sequence of up to 8 later chunks by itself, the wave together a longer one.
template <int NV>
struct alignas(16) Part {
  double v[NV];
};
template <int NV, int NT>
__device__ __forceinline__ void sum_sequences(const SeqArgs& a, const double* head, const double* seqp, double* tot) {
  static_assert(NV % 2 == 0, "16-byte parts");
  const Part<NV>* hp = reinterpret_cast<const Part<NV>*>(head);
  const int lane = threadIdx.x & 63;
  for (int s0 = (threadIdx.x >> 6) * 64; s0 < a.S; s0 += NT) {
    const int s = s0 + lane;
    int64_t b = 0, e = 0;
    if (s < a.S) {
      b = clip_tok(a.cu[s], a.N);
      e = clip_tok(a.cu[s + 1], a.N);
    }
    const bool any = e > b;
    const int64_t c0 = any ? b >> a.lg : 0, c1 = any ? (e - 1) >> a.lg : 0;
    Part<NV> v = {};
    if (any) v = reinterpret_cast<const Part<NV>*>(seqp)[s];
    const bool longer = c1 - c0 > 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 4 parts' loads in flight at a time
      if (longer || c0 + 4 * h >= c1) continue;
      Part<NV> x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = hp[min(c0 + 1 + 4 * h + k, c1)];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < NV; ++q) v.v[q] += c0 + 1 + 4 * h + k <= c1 ? x[k].v[q] : 0.0;
    }
    for (unsigned long long todo = __ballot(longer); todo; todo &= todo - 1) {
      const int l = __ffsll(todo) - 1;
      const int64_t cb = pick(c0, l) + 1, ce = pick(c1, l);
      double w[NV];
#pragma unroll
      for (int q = 0; q < NV; ++q) w[q] = 0.0;
#pragma unroll 4
      for (int64_t c = cb + lane; c <= ce; c += 64) {
        const Part<NV> x = hp[c];
#pragma unroll
        for (int q = 0; q < NV; ++q) w[q] += x.v[q];
      }
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        w[q] = wave_sum(w[q]);
        if (lane == l) v.v[q] += w[q];
      }
    }
    if (s < a.S) reinterpret_cast<Part<NV>*>(tot)[s] = v;
  }
}

// The sums of two values over the block's threads, to every thread; fixed
// order.
template <int NT>
__device__ __forceinline__ void block_sum2(double& x, double& y, double* red) {
  x = wave_sum(x);
  y = wave_sum(y);
  __syncthreads();  // red is free
  if ((threadIdx.x & 63) == 0) {
    red[2 * (threadIdx.x >> 6)] = x;
    red[2 * (threadIdx.x >> 6) + 1] = y;
  }
  __syncthreads();
  x = y = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    x += red[2 * w];
    y += red[2 * w + 1];
  }
}

// ---- preference ----
struct PrefArgs {
  int kind, average, P;
  double beta, eps;
  float* loss;
  float* pair_loss;
  float* rewards;
  float* coef;
};

__device__ __forceinline__ double softplus(double x) { return fmax(x, 0.0) + log1p(exp(-fabs(x))); }

template <int NT>
__device__ __forceinline__ void finish(const PrefArgs& p, int, const double* tot) {
  __shared__ double red[2 * NT / 64];
  double sum = 0.0, none = 0.0;
  for (int i = threadIdx.x; i < p.P; i += NT) {
    const double nc = tot[2 * (int64_t)i + 1], nr = tot[2 * ((int64_t)p.P + i) + 1];
    const double wc = p.average ? 1.0 / fmax(nc, 1.0) : 1.0, wr = p.average ? 1.0 / fmax(nr, 1.0) : 1.0;
    const double c = tot[2 * (int64_t)i] * wc, r = tot[2 * ((int64_t)p.P + i)] * wr;
    const double u = c - r, bu = p.beta * u;
    double l, du;
    if (p.kind == 0) {
      l = (1.0 - p.eps) * softplus(-bu);
      du = -(1.0 - p.eps) / (1.0 + exp(bu));
      if (p.eps > 0.0) {  // (a smoothed margin of infinite size: 0 * inf otherwise)
        l += p.eps * softplus(bu);
        du += p.eps / (1.0 + exp(-bu));
      }
      du *= p.beta;
    } else if (p.kind == 1) {
      l = bu != bu ? bu : fmax(1.0 - bu, 0.0);  // (fmax would drop a NaN)
      du = bu < 1.0 ? -p.beta : 0.0;
    } else {
      const double v = u - 0.5 / p.beta;
      l = v * v;
      du = 2.0 * v;
    }
    sum += l;
    p.pair_loss[i] = (float)l;
    p.rewards[i] = (float)(p.beta * c);
    p.rewards[p.P + i] = (float)(p.beta * r);
    p.coef[i] = (float)(du * wc / p.P);
    p.coef[p.P + i] = (float)(-du * wr / p.P);
  }
  block_sum2<NT>(sum, none, red);
  if (threadIdx.x == 0) *p.loss = (float)(sum / p.P);
}

// ---- policy ----
struct PolicyOut {
  int reduction;  // 0 mean over sequences of their mean, 1 mean over tokens, 2 sum / (S norm)
  double norm;
  float beta;
  float* loss;
  float* stats;
  float* weight;
};

template <int NT>
__device__ __forceinline__ void finish(const PolicyOut& p, int S, const double* tot) {
  __shared__ double red[2 * NT / 64];
  double tok = 0.0, cut = 0.0;
  for (int s = threadIdx.x; s < S; s += NT) {
    cut += tot[4 * (int64_t)s + 2];
    tok += tot[4 * (int64_t)s + 3];
  }
  block_sum2<NT>(tok, cut, red);
  double pol = 0.0, kl = 0.0;
  for (int s = threadIdx.x; s < S; s += NT) {
    const double* v = tot + 4 * (int64_t)s;
    const double w = p.reduction == 0   ? 1.0 / (S * fmax(v[3], 1.0))
                     : p.reduction == 1 ? 1.0 / fmax(tok, 1.0)
                                        : 1.0 / (S * p.norm);
    pol += w * v[0];
    kl += w * v[1];
    p.weight[s] = (float)w;
  }
  block_sum2<NT>(pol, kl, red);
  if (threadIdx.x == 0) {
    *p.loss = (float)(p.beta != 0.f ? pol + (double)p.beta * kl : pol);
    p.stats[0] = (float)pol;
    p.stats[1] = (float)kl;
    p.stats[2] = (float)(cut / fmax(tok, 1.0));
    p.stats[3] = (float)tok;
  }
}

constexpr int FT = 1024;  // threads of the finishing block

template <class Term>
__global__ void __launch_bounds__(256) seq_sum_kernel(const SeqArgs a, const Term term) {
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c < a.chunks) sum_chunk(a, term, c, threadIdx.x & 63, a.head, a.seqp);
}

template <class Term, class Out>
__global__ void __launch_bounds__(FT) seq_finish_kernel(const SeqArgs a, const Out out) {
  constexpr int NV = Term::NV;
  __shared__ alignas(16) double tot[SEQ_LDS * NV];
  if (a.S <= SEQ_LDS) {
    sum_sequences<NV, FT>(a, a.head, a.seqp, tot);
    __syncthreads();
    finish<FT>(out, a.S, tot);
  } else {
    sum_sequences<NV, FT>(a, a.head, a.seqp, a.seqp);
    __syncthreads();
    finish<FT>(out, a.S, a.seqp);
  }
}

// Few tokens and sequences: one block does both, the parts in LDS (the launch
// between them costs more than the tokens).
template <class Term, class Out>
__global__ void __launch_bounds__(FT) seq_small_kernel(const SeqArgs a, const Term term, const Out out) {
  constexpr int NV = Term::NV;
  __shared__ alignas(16) double tot[SEQ_LDS * NV];
  __shared__ alignas(16) double head[FT / 64 * NV];
  const int c = threadIdx.x >> 6;  // (at most FT / 64 chunks)
  if (c < a.chunks) sum_chunk(a, term, c, threadIdx.x & 63, head, tot);
  __syncthreads();
  sum_sequences<NV, FT>(a, head, tot, tot);
  __syncthreads();
  finish<FT>(out, a.S, tot);
}

template <class Term, class Out>
hipError_t run_seq(SeqArgs a, const Term& term, const Out& out, hipStream_t st) {
  if (a.N <= SEQ_SMALL && a.S <= SEQ_LDS) {
    // a chunk for every wave of the one block, of 64 tokens at least
    a.lg = 6;
    while ((int64_t(FT / 64) << a.lg) < a.N) ++a.lg;
    a.chunks = (a.N + (int64_t(1) << a.lg) - 1) >> a.lg;
    hipLaunchKernelGGL((seq_small_kernel<Term, Out>), dim3(1), dim3(FT), 0, st, a, term, out);
    return hipGetLastError();
  }
  if (a.chunks > 0) {
    hipLaunchKernelGGL((seq_sum_kernel<Term>), dim3((unsigned)((a.chunks + 3) / 4)), dim3(256), 0, st, a, term);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((seq_finish_kernel<Term, Out>), dim3(1), dim3(FT), 0, st, a, out);
  return hipGetLastError();
}

// ---- gradients: one wave per chunk, dlogp of every token of [0, N) ----
// payload 0: the sequence's coefficient or weight, 1: its advantage.
struct GradPay {
  static constexpr int NP = 2;
};

// f(raw, payload) of every counted token in a sequence, 0 elsewhere.
template <class Load, class F>
__device__ __forceinline__ void grad_chunk(const SeqArgs& a, const float* pay0, const float* pay1, float* dlogp,
                                           Load&& load, F&& f) {
  const int lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c >= a.chunks) return;
  const int64_t t0 = c << a.lg, t1 = min(t0 + (int64_t(1) << a.lg), a.N);
  Walk<GradPay> w;
  w.cu = a.cu;
  w.S = a.S;
  w.N = a.N;
  w.lane = lane;
  w.src[0] = pay0;
  w.src[1] = pay1;
  decltype(load(t0)) raw[UT];
  bool keep[UT];
  auto request = [&](int64_t p) {
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      const int64_t t = p + 64 * u + lane;
      const int64_t at = t < t1 ? t : t1 - 1;
      raw[u] = load(at);
      keep[u] = t < t1 && (!a.mask || a.mask[at]);
    }
  };
  request(t0);
  w.start(t0);
  for (int64_t p = t0; p < t1; p += STEP) {
    if (p > t0) request(p);
    const int64_t pe = min(p + STEP, t1);
    float d[UT];
#pragma unroll
    for (int u = 0; u < UT; ++u) d[u] = 0.f;
    for (int64_t pos = p; pos < pe;) {
      int64_t to, b;
      int l;
      if (w.next(pos, pe, to, b, l) >= 0) {
        const float q0 = pick(w.pay[0], l), q1 = pick(w.pay[1], l);
        const int lo = (int)(pos - p), hi = (int)(to - p);
#pragma unroll
        for (int u = 0; u < UT; ++u)
          if (64 * u < hi && 64 * u + 64 > lo) {  // (uniform)
            const float x = f(raw[u], q0, q1);
            if (keep[u] && 64 * u + lane >= lo && 64 * u + lane < hi) d[u] = x;
          }
      }
      pos = to;
    }
#pragma unroll
    for (int u = 0; u < UT; ++u) {
      const int64_t t = p + 64 * u + lane;
      if (t < t1) dlogp[t] = d[u];
    }
  }
}

__global__ void __launch_bounds__(256) pref_grad_kernel(const SeqArgs a, const float* __restrict__ coef,
                                                        const float* __restrict__ dloss, float* __restrict__ dlogp) {
  const float g = dloss ? *dloss : 1.f;
  grad_chunk(a, coef, nullptr, dlogp, [](int64_t) { return 0; }, [&](int, float q, float) { return g * q; });
}

__global__ void __launch_bounds__(256) policy_grad_kernel(const SeqArgs a, const PolicyArgs p,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ dloss, float* __restrict__ dlogp) {
  const float g = dloss ? *dloss : 1.f;
  grad_chunk(a, weight, p.adv_per_token ? nullptr : p.adv, dlogp, [&](int64_t t) { return p.load(t); },
             [&](const PolicyArgs::Raw& r, float w, float adv) {
               const PolicyTok k = policy_tok(p, r, adv);
               float d = 0.f;
               if (!k.cut && k.adv != 0.f) d = -k.ratio * k.adv;
               if (p.beta != 0.f) d -= p.beta * kl_slope((float)((double)r.ref - (double)r.lp));
               return g * w * d;
             });
}

SeqArgs seq_args(const LossSeqs& q, void* ws, int nv) {
  SeqArgs a;
  a.cu = q.cu;
  a.mask = q.mask;
  a.N = q.N;
  a.S = (int)q.S;
  a.lg = loss_chunk_log2(q.N);
  a.chunks = (q.N + (int64_t(1) << a.lg) - 1) >> a.lg;
  a.head = static_cast<double*>(ws);
  a.seqp = a.head + a.chunks * nv;
  return a;
}

PolicyArgs policy_args(const PolicyLossArgs& q) {
  PolicyArgs p;
  p.logp = q.logp;
  p.old = q.old;
  p.ref = q.ref;
  p.adv = q.adv;
  p.adv_per_token = q.adv_per_token;
  p.log_lo = log1p(-q.eps_low);
  p.log_hi = log1p(q.eps_high);
  p.r_lo = (float)(1.0 - q.eps_low);
  p.r_hi = (float)(1.0 + q.eps_high);
  p.beta = (float)q.beta;
  return p;
}

}  // namespace

// Tokens per wave: one step of 256 while that gives at most 8192 waves (all
// that are resident at once), then twice as many, up to 4096.
int loss_chunk_log2(int64_t N) {
  int lg = 8;
  while (lg < 12 && (N >> lg) > 8192) ++lg;
  return lg;
}

size_t loss_workspace(int64_t S, int64_t N, int nv) {
  const int lg = loss_chunk_log2(N);
  return (size_t)(((N + (int64_t(1) << lg) - 1) >> lg) + S) * nv * sizeof(double);
}

hipError_t launch_pref_loss(const LossSeqs& q, const PrefLossArgs& l, void* ws, hipStream_t st) {
  const SeqArgs a = seq_args(q, ws, PrefTerm::NV);
  const PrefTerm term{l.logp, l.ref};
  const PrefArgs out{l.kind, l.average, (int)(q.S / 2), l.beta, l.eps, l.loss, l.pair_loss, l.rewards, l.coef};
  return run_seq(a, term, out, st);
}

hipError_t launch_pref_grad(const LossSeqs& q, const float* coef, const float* dloss, float* dlogp, hipStream_t st) {
  const SeqArgs a = seq_args(q, nullptr, PrefTerm::NV);
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(pref_grad_kernel, dim3((unsigned)((a.chunks + 3) / 4)), dim3(256), 0, st, a, coef, dloss, dlogp);
  return hipGetLastError();
}

hipError_t launch_policy_loss(const LossSeqs& q, const PolicyLossArgs& l, void* ws, hipStream_t st) {
  const SeqArgs a = seq_args(q, ws, PolicyTerm::NV);
  const PolicyTerm term{policy_args(l)};
  const PolicyOut out{l.reduction, l.norm, (float)l.beta, l.loss, l.stats, l.weight};
  return run_seq(a, term, out, st);
}

hipError_t launch_policy_grad(const LossSeqs& q, const PolicyLossArgs& l, const float* dloss, float* dlogp,
                              hipStream_t st) {
  const SeqArgs a = seq_args(q, nullptr, PolicyTerm::NV);
  if (a.chunks == 0) return hipSuccess;
  hipLaunchKernelGGL(policy_grad_kernel, dim3((unsigned)((a.chunks + 3) / 4)), dim3(256), 0, st, a, policy_args(l),
                     l.weight, dloss, dlogp);
  return hipGetLastError();
}

}  // namespace lora
