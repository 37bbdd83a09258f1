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

// 16 bytes of a row whose address is a multiple of the element size only
// (rows of an odd vocabulary): one global_load_dwordx4 either way.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
struct Row;
template <>
struct Row<uint16_t> {  // bf16 bit patterns
  static constexpr int E = 8;
  typedef u32x4_e2 V;
  static __device__ __forceinline__ float at(const uint16_t* p) { return __builtin_bit_cast(float, (uint32_t)*p << 16); }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }
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
// sum s of e^(tau (z - m)); logp = tau (z_t - m) - log s.  m and log s are
// kept apart (their sum, the log-sum-exp, would round away what a confident
// row's small log-probability is made of).
// ---------------------------------------------------------------------------
__device__ __forceinline__ float fexp2(float x) { return __builtin_amdgcn_exp2f(x); }

// (m, s) of two parts of a row; a part with no finite value has m = -inf,
// s = 0 and adds nothing.  c = tau log2 e.
__device__ __forceinline__ void join_max_sum(float& m, float& s, float m2, float s2, float c) {
  const float nm = fmaxf(m, m2), base = nm == -INFINITY ? 0.f : nm;
  s = s * fexp2((m - base) * c) + s2 * fexp2((m2 - base) * c);
  m = nm;
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) token_logp_kernel(const T* __restrict__ z, int64_t ld, int64_t rows, int V,
                                                        const int64_t* __restrict__ target, float tau,
                                                        float* __restrict__ logp, float* __restrict__ stats) {
  using R = Row<T>;
  constexpr int E = R::E, U = 4;
  __shared__ float red[2][NT / 64];
  const float c = tau * LOG2E;
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* zr = z + row * ld;
    const int64_t t = target[row];
    const bool has = t >= 0 && t < V;
    const float zt = has ? R::at(zr + t) : 0.f;
    float m = -INFINITY, s = 0.f;
    auto take = [&](const u32x4 v) {
      float x[E];
      R::unpack(v, x);
      float cm = x[0];
#pragma unroll
      for (int e = 1; e < E; ++e) cm = fmaxf(cm, x[e]);
      const float nm = fmaxf(m, cm), base = nm == -INFINITY ? 0.f : nm;
      s *= fexp2((m - base) * c);
#pragma unroll
      for (int e = 0; e < E; ++e) s += fexp2((x[e] - base) * c);
      m = nm;
    };
    const int nv = V / E;
    int i = tid;
    for (; i + (U - 1) * NT < nv; i += U * NT) {
      u32x4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const typename R::V*>(zr + (int64_t)(i + u * NT) * E);
#pragma unroll
      for (int u = 0; u < U; ++u) take(v[u]);
    }
    for (; i < nv; i += NT) take(*reinterpret_cast<const typename R::V*>(zr + (int64_t)i * E));
    if (tid < V - nv * E) join_max_sum(m, s, R::at(zr + (int64_t)nv * E + tid), 1.f, c);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
      join_max_sum(m, s, m2, s2, c);
    }
    if constexpr (NT > 64) {
      if ((tid & 63) == 0) {
        red[0][tid >> 6] = m;
        red[1][tid >> 6] = s;
      }
      __syncthreads();
      m = red[0][0];
      s = red[1][0];
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) join_max_sum(m, s, red[0][w], red[1][w], c);
    }
    if (tid == 0) {
      const float ls = logf(s);
      logp[row] = has ? (zt - m) * tau - ls : 0.f;
      stats[2 * row] = m;
      stats[2 * row + 1] = ls;
    }
    if constexpr (NT > 64) __syncthreads();  // red is free for the next row
  }
}

// dz_j = g tau (1[j = t] - e^(tau (z_j - m) - log s)).  A row without a token
// or with g = 0 is not read: its gradient is zero whatever it holds.  dz may
// be z (every thread reads its elements before it writes them).
constexpr int GRAD_U = 4, GRAD_NT = 256;

template <typename T>
__global__ void __launch_bounds__(GRAD_NT) token_logp_grad_kernel(const T* z, int64_t ld, int64_t rows, int V, int segs,
                                                                  const int64_t* __restrict__ target, float tau,
                                                                  const float* __restrict__ stats,
                                                                  const float* __restrict__ dlogp, T* dz,
                                                                  int64_t ldd) {
  using R = Row<T>;
  constexpr int E = R::E, U = GRAD_U, NT = GRAD_NT;
  const int nv = V / E;
  const int64_t items = rows * segs;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / segs;
    const int seg = (int)(it - row * segs);
    const int64_t t = target[row];
    const float g = t >= 0 && t < V ? dlogp[row] * tau : 0.f;
    const T* zr = z + row * ld;
    T* dr = dz + row * ldd;
    const bool zero = g == 0.f;
    const float m = stats[2 * row], ls2 = stats[2 * row + 1] * LOG2E, c = tau * LOG2E;
    auto grad = [&](float x, int64_t j) { return (j == t ? g : 0.f) - g * fexp2((x - m) * c - ls2); };
    const int i0 = seg * (U * NT) + threadIdx.x;
    u32x4 v[U];
    if (!zero) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * NT < nv) v[u] = *reinterpret_cast<const typename R::V*>(zr + (int64_t)(i0 + u * NT) * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = (int64_t)(i0 + u * NT) * E;
      if (i0 + u * NT >= nv) continue;
      u32x4 o = {0u, 0u, 0u, 0u};
      if (!zero) {
        float x[E];
        R::unpack(v[u], x);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = grad(x[e], j + e);
        o = R::pack(x);
      }
      *reinterpret_cast<typename R::V*>(dr + j) = o;
    }
    // the row's last V % E elements: the last segment's first threads
    if (seg == segs - 1 && (int)threadIdx.x < V - nv * E) {
      const int64_t j = (int64_t)nv * E + threadIdx.x;
      R::put(dr + j, zero ? 0.f : grad(R::at(zr + j), j));
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
  if (V <= 2048) return go(std::integral_constant<int, 64>{});
  if (rows >= 1024) return go(std::integral_constant<int, 256>{});
  return go(std::integral_constant<int, 1024>{});
}

template <typename T>
hipError_t run_logp_grad(const T* z, int64_t ld, int64_t rows, int64_t V, const int64_t* target, float tau,
                         const float* stats, const float* dlogp, T* dz, int64_t ldd, hipStream_t st) {
  const int64_t per = (int64_t)GRAD_U * GRAD_NT * Row<T>::E;
  const int64_t segs = std::max<int64_t>(1, (V + per - 1) / per);
  const unsigned grid = (unsigned)std::min<int64_t>(rows * segs, 1 << 22);
  hipLaunchKernelGGL((token_logp_grad_kernel<T>), dim3(grid), dim3(GRAD_NT), 0, st, z, ld, rows, (int)V, (int)segs,
                     target, tau, stats, dlogp, dz, ldd);
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
// ones), finds the first of them by a 64-way search and leaves
//   seqp[s]: the part of sequence s in the chunk it starts in,
//   head[c]: the part in chunk c of a sequence that started before it;
// a sequence's sum is seqp[s] plus head[c] over the later chunks it reaches,
// always in that order.  Sums are held in 64 bits: a preference margin is the
// difference of two sums over thousands of tokens.
// cu is read on the device and cannot be checked before the launch: every
// index that comes from it is clipped to [0, N], and tokens outside
// [cu[0], cu[S]) belong to no sequence.
// ---------------------------------------------------------------------------
namespace {

__device__ __forceinline__ int64_t clip_tok(int64_t t, int64_t N) { return t < 0 ? 0 : (t > N ? N : t); }

// The number of sequences that end at or before token t (the first that ends
// after it), by the whole wave.
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

// f(s, b, lo, hi): every stretch [lo, hi) of tokens of [t0, t1) that lies in
// one sequence s (which starts at b), in order; called by the whole wave with
// uniform arguments.  gap(lo, hi): a stretch in no sequence.
template <class F, class G>
__device__ __forceinline__ void walk_chunk(const int64_t* cu, int S, int64_t N, int64_t t0, int64_t t1, int lane, F&& f,
                                           G&& gap) {
  int base = first_seq(cu, S, t0, lane);
  int64_t pos = t0;
  // lane l holds the end of sequence base + l
  while (base < S && pos < t1) {
    const bool in = base + lane < S;
    const int64_t end = in ? clip_tok(cu[base + lane + 1], N) : 0;
    int64_t beg0 = clip_tok(cu[base], N);
    unsigned long long todo;
    while (pos < t1 && (todo = __ballot(in && end > pos)) != 0) {
      const int l = __ffsll(todo) - 1;
      const int64_t prev = __shfl(end, l > 0 ? l - 1 : 0);
      const int64_t b = l > 0 ? prev : beg0, e = __shfl(end, l);
      if (b > pos) {  // before the first sequence
        const int64_t to = b < t1 ? b : t1;
        gap(pos, to);
        pos = to;
        continue;
      }
      const int64_t to = e < t1 ? e : t1;
      f(base + l, b, pos, to);
      pos = to;
    }
    base += 64;
  }
  if (pos < t1) gap(pos, t1);  // behind the last sequence
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// preference: the log-ratios and the number of counted tokens
struct PrefTerm {
  static constexpr int NV = 2;
  const float* logp;
  const float* ref;
  __device__ __forceinline__ void add(int64_t t, int, double (&v)[NV]) const {
    v[0] += ref ? (double)logp[t] - (double)ref[t] : (double)logp[t];
    v[1] += 1.0;
  }
};

// e^d - d - 1: its series where the three cancel (the rest is below 2e-9 of
// the sum there), else from expm1
__device__ __forceinline__ float kl_term(float d) {
  if (fabsf(d) < 0.25f) {
    const float q =
        0.5f + d * (1.f / 6 + d * (1.f / 24 + d * (1.f / 120 + d * (1.f / 720 + d * (1.f / 5040 + d / 40320)))));
    return d * d * q;
  }
  return expm1f(d) - d;
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
};

// The clip borders are compared on logp - old in 64 bits, where the difference
// of two fp32 values is exact: a ratio rounded to fp32 first could fall on the
// other side of its border.
struct PolicyTok {
  float ratio, adv;
  bool cut;  // the clipped branch holds: no gradient through the ratio
};
__device__ __forceinline__ PolicyTok policy_tok(const PolicyArgs& p, int64_t t, int s) {
  PolicyTok k;
  k.adv = p.adv[p.adv_per_token ? t : (int64_t)s];
  const double d = p.old ? (double)p.logp[t] - (double)p.old[t] : 0.0;
  const bool over = k.adv > 0.f && d > p.log_hi, under = k.adv < 0.f && d < p.log_lo;
  k.cut = over || under;
  k.ratio = over ? p.r_hi : (under ? p.r_lo : expf((float)d));
  return k;
}

struct PolicyTerm {
  static constexpr int NV = 4;
  PolicyArgs p;
  __device__ __forceinline__ void add(int64_t t, int s, double (&v)[NV]) const {
    const PolicyTok k = policy_tok(p, t, s);
    v[0] += k.adv == 0.f ? 0.0 : -((double)k.ratio * (double)k.adv);
    if (p.ref) v[1] += (double)kl_term((float)((double)p.ref[t] - (double)p.logp[t]));
    v[2] += k.cut ? 1.0 : 0.0;
    v[3] += 1.0;
  }
};

struct SeqArgs {
  const int64_t* cu;
  const uint8_t* mask;
  int64_t N;
  int S, ch;
  int64_t chunks;
  double* head;  // [chunks][NV]
  double* seqp;  // [S][NV]; then the sequences' sums
};

template <class Term>
__device__ __forceinline__ void sum_chunk(const SeqArgs& a, const Term& term, int64_t c, int lane) {
  constexpr int NV = Term::NV;
  const int64_t t0 = c * a.ch, t1 = min(t0 + a.ch, a.N);
  walk_chunk(
      a.cu, a.S, a.N, t0, t1, lane,
      [&](int s, int64_t b, int64_t lo, int64_t hi) {
        double v[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] = 0.0;
#pragma unroll 4
        for (int64_t t = lo + lane; t < hi; t += 64)
          if (!a.mask || a.mask[t]) term.add(t, s, v);
        double* out = b < t0 ? a.head + c * NV : a.seqp + (int64_t)s * NV;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          v[q] = wave_sum(v[q]);
          if (lane == 0) out[q] = v[q];
        }
      },
      [](int64_t, int64_t) {});
}

// seqp[s] = the sum of sequence s, for every s (one block): a lane takes a
// sequence of up to 8 later chunks by itself, the wave together a longer one.
template <int NV, int NT>
__device__ __forceinline__ void sum_sequences(const SeqArgs& a) {
  const int lane = threadIdx.x & 63;
  for (int s0 = (threadIdx.x >> 6) * 64; s0 < a.S; s0 += NT) {
    const int s = s0 + lane;
    int64_t b = 0, e = 0;
    if (s < a.S) {
      b = clip_tok(a.cu[s], a.N);
      e = clip_tok(a.cu[s + 1], a.N);
    }
    const bool any = e > b;
    const int64_t c0 = any ? b / a.ch : 0, c1 = any ? (e - 1) / a.ch : 0;
    double v[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) v[q] = any ? a.seqp[(int64_t)s * NV + q] : 0.0;
    const bool longer = c1 - c0 > 8;
    if (!longer)
      for (int64_t c = c0 + 1; c <= c1; ++c)
#pragma unroll
        for (int q = 0; q < NV; ++q) v[q] += a.head[c * NV + q];
    for (unsigned long long todo = __ballot(longer); todo; todo &= todo - 1) {
      const int l = __ffsll(todo) - 1;
      const int64_t cb = __shfl(c0, l) + 1, ce = __shfl(c1, l);
      double w[NV];
#pragma unroll
      for (int q = 0; q < NV; ++q) w[q] = 0.0;
      for (int64_t c = cb + lane; c <= ce; c += 64)
#pragma unroll
        for (int q = 0; q < NV; ++q) w[q] += a.head[c * NV + q];
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        w[q] = wave_sum(w[q]);
        if (lane == l) v[q] += w[q];
      }
    }
    if (s < a.S)
#pragma unroll
      for (int q = 0; q < NV; ++q) a.seqp[(int64_t)s * NV + q] = v[q];
  }
}

// The sum over the block's threads, to every thread; fixed order.
template <int NT>
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = wave_sum(v);
  __syncthreads();  // red is free
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t += red[w];
  return t;
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
__device__ __forceinline__ void pref_finish(const SeqArgs& a, const PrefArgs& p) {
  __shared__ double red[NT / 64];
  double sum = 0.0;
  for (int i = threadIdx.x; i < p.P; i += NT) {
    const double nc = a.seqp[2 * (int64_t)i + 1], nr = a.seqp[2 * ((int64_t)p.P + i) + 1];
    const double wc = p.average ? 1.0 / fmax(nc, 1.0) : 1.0, wr = p.average ? 1.0 / fmax(nr, 1.0) : 1.0;
    const double c = a.seqp[2 * (int64_t)i] * wc, r = a.seqp[2 * ((int64_t)p.P + i)] * wr;
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
  sum = block_sum<NT>(sum, red);
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
__device__ __forceinline__ void policy_finish(const SeqArgs& a, const PolicyOut& p) {
  __shared__ double red[NT / 64];
  double tok = 0.0, cut = 0.0;
  for (int s = threadIdx.x; s < a.S; s += NT) {
    cut += a.seqp[4 * (int64_t)s + 2];
    tok += a.seqp[4 * (int64_t)s + 3];
  }
  tok = block_sum<NT>(tok, red);
  cut = block_sum<NT>(cut, red);
  double pol = 0.0, kl = 0.0;
  for (int s = threadIdx.x; s < a.S; s += NT) {
    const double* v = a.seqp + 4 * (int64_t)s;
    const double w = p.reduction == 0   ? 1.0 / (a.S * fmax(v[3], 1.0))
                     : p.reduction == 1 ? 1.0 / fmax(tok, 1.0)
                                        : 1.0 / (a.S * p.norm);
    pol += w * v[0];
    kl += w * v[1];
    p.weight[s] = (float)w;
  }
  pol = block_sum<NT>(pol, red);
  kl = block_sum<NT>(kl, red);
  if (threadIdx.x == 0) {
    *p.loss = (float)(p.beta != 0.f ? pol + (double)p.beta * kl : pol);
    p.stats[0] = (float)pol;
    p.stats[1] = (float)kl;
    p.stats[2] = (float)(cut / fmax(tok, 1.0));
    p.stats[3] = (float)tok;
  }
}

__device__ __forceinline__ void finish(const SeqArgs& a, const PrefArgs& p) { pref_finish<1024>(a, p); }
__device__ __forceinline__ void finish(const SeqArgs& a, const PolicyOut& p) { policy_finish<1024>(a, p); }

template <class Term>
__global__ void __launch_bounds__(256) seq_sum_kernel(const SeqArgs a, const Term term) {
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c < a.chunks) sum_chunk(a, term, c, threadIdx.x & 63);
}

template <class Term, class Out>
__global__ void __launch_bounds__(1024) seq_finish_kernel(const SeqArgs a, const Out out) {
  sum_sequences<Term::NV, 1024>(a);
  __syncthreads();
  finish(a, out);
}

// Few tokens: one block does both (the launch between them costs more than
// the tokens).
template <class Term, class Out>
__global__ void __launch_bounds__(1024) seq_small_kernel(const SeqArgs a, const Term term, const Out out) {
  for (int64_t c = threadIdx.x >> 6; c < a.chunks; c += 16) sum_chunk(a, term, c, threadIdx.x & 63);
  __syncthreads();
  sum_sequences<Term::NV, 1024>(a);
  __syncthreads();
  finish(a, out);
}

template <class Term, class Out>
hipError_t run_seq(const SeqArgs& a, const Term& term, const Out& out, hipStream_t st) {
  if (a.N <= SEQ_SMALL) {
    hipLaunchKernelGGL((seq_small_kernel<Term, Out>), dim3(1), dim3(1024), 0, st, a, term, out);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((seq_sum_kernel<Term>), dim3((unsigned)((a.chunks + 3) / 4)), dim3(256), 0, st, a, term);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((seq_finish_kernel<Term, Out>), dim3(1), dim3(1024), 0, st, a, out);
  return hipGetLastError();
}

// ---- gradients: one wave per chunk, dlogp of every token of [0, N) ----
__global__ void __launch_bounds__(256) pref_grad_kernel(const SeqArgs a, const float* __restrict__ coef,
                                                        const float* __restrict__ dloss, float* __restrict__ dlogp) {
  const int lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c >= a.chunks) return;
  const int64_t t0 = c * a.ch, t1 = min(t0 + a.ch, a.N);
  const float g = dloss ? *dloss : 1.f;
  walk_chunk(
      a.cu, a.S, a.N, t0, t1, lane,
      [&](int s, int64_t, int64_t lo, int64_t hi) {
        const float w = g * coef[s];
#pragma unroll 4
        for (int64_t t = lo + lane; t < hi; t += 64) dlogp[t] = (!a.mask || a.mask[t]) ? w : 0.f;
      },
      [&](int64_t lo, int64_t hi) {
        for (int64_t t = lo + lane; t < hi; t += 64) dlogp[t] = 0.f;
      });
}

__global__ void __launch_bounds__(256) policy_grad_kernel(const SeqArgs a, const PolicyArgs p,
                                                          const float* __restrict__ weight,
                                                          const float* __restrict__ dloss, float* __restrict__ dlogp) {
  const int lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (c >= a.chunks) return;
  const int64_t t0 = c * a.ch, t1 = min(t0 + a.ch, a.N);
  const float g = dloss ? *dloss : 1.f;
  walk_chunk(
      a.cu, a.S, a.N, t0, t1, lane,
      [&](int s, int64_t, int64_t lo, int64_t hi) {
        const float w = g * weight[s];
#pragma unroll 4
        for (int64_t t = lo + lane; t < hi; t += 64) {
          float d = 0.f;
          if (!a.mask || a.mask[t]) {
            const PolicyTok k = policy_tok(p, t, s);
            if (!k.cut && k.adv != 0.f) d = -k.ratio * k.adv;
            if (p.beta != 0.f) d -= p.beta * expm1f((float)((double)p.ref[t] - (double)p.logp[t]));
            d *= w;
          }
          dlogp[t] = d;
        }
      },
      [&](int64_t lo, int64_t hi) {
        for (int64_t t = lo + lane; t < hi; t += 64) dlogp[t] = 0.f;
      });
}

SeqArgs seq_args(const LossSeqs& q, void* ws, int nv) {
  SeqArgs a;
  a.cu = q.cu;
  a.mask = q.mask;
  a.N = q.N;
  a.S = (int)q.S;
  a.ch = loss_chunk(q.N);
  a.chunks = (q.N + a.ch - 1) / a.ch;
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

// Tokens per wave: about 2048 waves (two per SIMD), at least a wave's 4 rounds
// of 64 and at most 4096.
int loss_chunk(int64_t N) {
  const int64_t c = ((N + 2047) / 2048 + 63) / 64 * 64;
  return (int)std::min<int64_t>(4096, std::max<int64_t>(256, c));
}

size_t loss_workspace(int64_t S, int64_t N, int nv) {
  const int64_t ch = loss_chunk(N);
  return (size_t)((N + ch - 1) / ch + S) * nv * sizeof(double);
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
