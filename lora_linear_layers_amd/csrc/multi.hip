// multi.hip - a projection whose rows each carry an adapter of their own:
//
//     y_t = W x_t + s_a B_a (A_a x_t),   a = index[t]   (none: y_t = W x_t)
//
// for batches of requests that share a base weight (decode steps and packed
// prompts) and for training several adapters at once; with its gradients
//
//     dX_t = W^T dy_t + s_a A_a^T (B_a^T dy_t)
//     dB_a = s_a sum_{t in a} dy_t (A_a x_t)^T,  dA_a = s_a sum_{t in a} (B_a^T dy_t) x_t^T
//
// The layer of one adapter adds the panel P = s X A^T, a rank-r strip, as a
// second segment to the base product's contraction.  Here the strip holds
// each row's own adapter's columns, P [M, r], and the segment of a tile of rows
// is made of the adapters that its rows carry, one after the other: row t has
// its strip in its adapter's columns and zeros in the others' (offsets past
// the buffer give those zeros: nothing is expanded in memory).  Rows need no order.
// In the order of a batch (a request's tokens together) a tile carries a few
// adapters, a 64-column stage for 64 / r of them beside the base's d_in / 64
// stages; in any order it stays right, at a stage for each 64 / r of the adapters it
// meets.  The gradients contract, per 64 rows of the stacked adapters, the
// 64-token tiles in which one of them occurs (again a list).
//
// bf16 runs on the layer's own MFMA kernels with those lists (gemm_w4_half.h,
// gemm_w4_stream.h, gemm_panel.h); fp32 on the simple kernels below.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_panel.h"
#include "gemm_w4_half.h"
#include "gemm_w4_stream.h"
#include "launch.h"

namespace lora {

namespace {

template <typename T>
__device__ __forceinline__ float val(T x) {
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(float, (uint32_t)x << 16);
  else
    return x;
}

__device__ __forceinline__ int adapter_at(const int* index, int64_t t, int64_t M, int n) {
  const int a = t < M ? index[t] : -1;
  return a >= 0 && a < n ? a : -1;
}

// ---------------------------------------------------------------------------
// lists.  Blocks [0, T128): the adapters of a 128-row tile, in the order of
// their first rows; then T256 blocks, of a 256-row tile; then the row groups of
// the gradients: the 64-token tiles in which an adapter of the group occurs.
// The first block also clears the stream kernel's counters.  Then `chunks` blocks
// an adapter, which look for infinities and NaNs in their part of its second
// operand if a row carries it: one adapter's must not reach the others' rows; and the
// backward's transposes of the stacks.  One launch, 7 to 8 us at 4001 rows of 32 adapters or
// 8192 of 8: what its longest blocks wait for, the indexes and then a share of an operand.
// ---------------------------------------------------------------------------
// The distinct values >= 0 of a wave's 64, in the order of their first lanes:
// lane k < the returned number gets the k-th.
__device__ __forceinline__ int wave_distinct(int v, int lane, int& mine) {
  uint64_t left = __ballot(v >= 0);
  int k = 0;
  mine = -1;
  while (left) {
    const int x = __builtin_amdgcn_readlane(v, __builtin_ctzll(left));
    left &= ~__ballot(v == x);
    mine = lane == k ? x : mine;
    ++k;
  }
  return k;
}

// dst [n][C, R] = src [n][R, C] (bf16) transposed, block b of its 64 x 32 tiles
// (64 along C): rows in 8-byte pieces on both sides (R and C multiples of 8).
__device__ __forceinline__ void transpose_stack(const MultiTranspose& q, int64_t b, uint16_t (*tile)[36]) {
  const int64_t tc = (q.C + 63) / 64, per = tc * ((q.R + 31) / 32), z = b / per, id = b - z * per;
  const int64_t r0 = id / tc * 32, c0 = id % tc * 64;
  const uint16_t* src = static_cast<const uint16_t*>(q.src) + z * q.R * q.C;
  uint16_t* dst = static_cast<uint16_t*>(q.dst) + z * q.R * q.C;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 16 rows of 16 pieces a pass
    const int rr = (threadIdx.x >> 4) + 16 * h, cc = (threadIdx.x & 15) * 4;
    if (r0 + rr < q.R && c0 + cc < q.C) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(src + (r0 + rr) * q.C + c0 + cc);
#pragma unroll
      for (int e = 0; e < 4; ++e) tile[cc + e][rr] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // 32 columns of 8 pieces a pass
    const int cc = (threadIdx.x >> 3) + 32 * h, rr = (threadIdx.x & 7) * 4;
    if (c0 + cc < q.C && r0 + rr < q.R)
      *reinterpret_cast<u32x2*>(dst + (c0 + cc) * q.R + r0 + rr) = *reinterpret_cast<const u32x2*>(&tile[cc][rr]);
  }
}

__global__ void __launch_bounds__(256) multi_lists_kernel(const MultiLists q) {
  __shared__ int ids[256];
  __shared__ __attribute__((aligned(8))) uint16_t tile[64][36];
  __shared__ int wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int b = blockIdx.x;
  if (b == 0)
    for (int i = tid; i < q.nzero; i += 256) q.zero[i] = 0;
  // positions of the threads with `keep` among those before them, and their number
  auto place = [&](bool keep, int& count) {
    const uint64_t m = __ballot(keep);
    __syncthreads();
    if (lane == 0) wsum[wave] = __popcll(m);
    __syncthreads();
    int before = 0;
    count = 0;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) before += wsum[w];
      count += wsum[w];
    }
    return before + __popcll(m & ((1ull << lane) - 1));
  };
  if (b < q.t128 + q.t256) {
    const int rows = b < q.t128 ? 128 : 256;
    const int tile = b < q.t128 ? b : b - q.t128;
    int* list = (b < q.t128 ? q.list128 : q.list256) + (int64_t)tile * q.cap(rows);
    int* cnt = (b < q.t128 ? q.cnt128 : q.cnt256) + tile;
    const int a = tid < rows ? adapter_at(q.index, (int64_t)tile * rows + tid, q.M, q.n) : -1;
    // each wave's own, then those that no wave before it has
    int mine;
    const int k = wave_distinct(a, lane, mine);
    ids[tid] = mine;
    if (lane == 0) wsum[wave] = k;
    __syncthreads();
    bool keep = lane < k;
    for (int w = 0; w < wave; ++w)
      for (int e = 0; e < wsum[w]; ++e) keep = keep && ids[64 * w + e] != mine;
    int count;
    const int at = place(keep, count);
    if (keep) list[at] = mine;
    if (tid == 0) *cnt = count;
    return;
  }
  b -= q.t128 + q.t256;
  if (b >= q.groups + q.n * q.chunks) {
    const int64_t k = b - (q.groups + (int64_t)q.n * q.chunks);
    transpose_stack(q.tr[k >= q.tr0 ? 1 : 0], k >= q.tr0 ? k - q.tr0 : k, tile);
    return;
  }
  if (b >= q.groups) {
    b -= q.groups;
    const int a = b / q.chunks, c = b - a * q.chunks;
    int any = 0;
#pragma unroll 16
    for (int64_t t = tid; t < q.M; t += 256) any |= q.index[t] == a;
    if (!__syncthreads_or(any)) {
      if (tid == 0) q.bad[b] = 0;
      return;
    }
    const int64_t end = min((int64_t)(c + 1) * q.pieces, q.scan16);
    const u32x4* v = reinterpret_cast<const u32x4*>(q.scan) + (int64_t)a * q.scan16;
    uint32_t found = 0;
#pragma unroll 8
    for (int64_t i = (int64_t)c * q.pieces + tid; i < end; i += 256) {
      const u32x4 x = v[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        found |= (x[k] & 0x7F80u) == 0x7F80u;
        found |= (x[k] & 0x7F800000u) == 0x7F800000u;
      }
    }
    const int bad = __syncthreads_or((int)found);
    if (tid == 0) q.bad[b] = bad ? 1 : 0;
    return;
  }
  // row group: adapters [lo, hi).  A wave's 64 tokens are a tile; 256 tiles a round
  const int lo = b * q.per, hi = min(lo + q.per, q.n);
  const int64_t t64 = (q.M + 63) / 64;
  int* list = q.glist + (int64_t)b * t64;
  int n = 0;
  for (int64_t base = 0; base < t64; base += 256) {
    const int steps = (int)min((t64 - base + 3) / 4, (int64_t)64);
    __syncthreads();
    ids[tid] = 0;
    __syncthreads();
#pragma unroll 16
    for (int i = 0; i < steps; ++i) {
      const int64_t t = (base + 4 * i) * 64 + tid;
      const int a = t < q.M ? q.index[t] : -1;
      if (__ballot(a >= lo && a < hi) && lane == 0) ids[4 * i + wave] = 1;
    }
    __syncthreads();
    int count;
    const bool mine = ids[tid] != 0;
    const int at = place(mine, count);
    if (mine) list[n + at] = (int)(base + tid);
    n += count;
  }
  if (tid == 0) q.gcnt[b] = n;
}

// ---------------------------------------------------------------------------
// strips
// ---------------------------------------------------------------------------
// bf16: partials of the tile's strips (gemm_panel.h), 64 columns of its adapters
// after the other, dealt to gridDim.z blocks.  (A block for every 64 columns that a
// tile could have, most of which leave at once, cost 5 of 16 us with 32 adapters:
// each takes a CU's LDS for its launch.)  Two panels in one launch (the backward's
// P and Q): splits [0, s0) of the grid are the first one's.
// A stream of X, as the layer's own panel: 8192 x 4096 twice (P and Q) in 58 us, 4001 x
// 4096 in 16, 2048 x 4096 in 12.  Rows in random order read X again for every 64 columns of their tile's
// adapters (64 of rank 16: 14 times, 525 us).
__global__ void __launch_bounds__(pdma::NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
multi_panel_kernel(const GemmPair q) {
  const int y = (int)blockIdx.y, w = y >= q.s0 ? 1 : 0;
  __shared__ __attribute__((aligned(1024))) char smem[pdma::Cfg<PANEL_BM, 64>::LDS];
  const GemmArgs& p = q.g[w];
  const int mt = blockIdx.x, cols = scalar_at(p.ad_cnt, mt) * p.ad_r;
  for (int cg = blockIdx.z; 64 * cg < cols; cg += gridDim.z) {
    panel_dma_tile<PANEL_BM, 64, true>(smem, p, mt, w ? y - q.s0 : y, cg);
    __syncthreads();  // (the ring is free again)
  }
}

// The strips of a 64-token tile from their partials, bf16(s_a sum), of one or
// both operands: `P` [M, r] for the product (NaNs for a row whose adapter's
// second operand is spoilt, which its tiles' lists are told here), and, for the
// gradients, `Pt` [n r, M8]: the strips spread over their group's rows, zeros
// where a token has another adapter, for the groups that the tile meets.  A token
// with an infinity or NaN in a strip (its own row of X or dY has one then) would
// reach the other adapters of its group as zero times that: its strips are zeros
// there, its bit in `mask` is clear like that of a token without adapter, and
// its adapter's gradients are NaNs (gbad).  The strips are rounded to bf16 here, as the
// layer's panel is, for the matrix cores: 2^-9 of a strip, next to the output's own
// rounding.  6 to 7 us at 8192 tokens of 8 adapters, the latency of index, partials and stores;
// a token's thread reads its adapter's flags (MultiLists::bad) one after the other, which is
// most of it where few adapters have much data and so many flags: 4001 rows, d_out 14336,
// 8 adapters of 16 (28 flags) 5.5 us, 2 of 64 (112) 14, one of 128 (224) 25.
__global__ void __launch_bounds__(256) multi_strip_kernel(const MultiStrip s) {
  __shared__ int ids[64], spoilt[64], bad[64], groups[64];
  __shared__ float sc[64];
  __shared__ int ngroups;
  __shared__ __attribute__((aligned(16))) uint16_t v[2][64 * (kMultiMaxRank + 4)];
  const int tid = threadIdx.x, r = s.r, pitch = r + 4;
  const int64_t t0 = (int64_t)blockIdx.x * 64;
  auto is_bad = [&](int a) {
    int b = 0;
    for (int c = 0; c < s.chunks; ++c) b |= s.bad[(int64_t)a * s.chunks + c];
    return b;
  };
  if (tid < 64) {
    const int a = adapter_at(s.index, t0 + tid, s.M, s.n);
    ids[tid] = a;
    spoilt[tid] = 0;
    sc[tid] = a >= 0 ? s.scales[a] : 0.f;
    bad[tid] = a >= 0 && s.chunks ? is_bad(a) : 0;
    int g;
    const int k = wave_distinct(a >= 0 ? a / s.per : -1, tid, g);
    if (tid < k) groups[tid] = g;
    if (tid == 0) ngroups = k;
  } else if (s.chunks && tid >= 192) {
    // the lists that this block's tile starts
    auto mark = [&](int* list, int count) {
      for (int e = tid - 192; e < count; e += 64)
        if (is_bad(list[e])) list[e] |= (int)AD_BAD;
    };
    const int b = blockIdx.x;
    if (s.list128 && b % 2 == 0) mark(s.list128 + (int64_t)(b / 2) * min(s.n, 128), s.cnt128[b / 2]);
    if (s.list256 && b % 4 == 0) mark(s.list256 + (int64_t)(b / 4) * min(s.n, 256), s.cnt256[b / 4]);
  }
  __syncthreads();
  const int r4 = r >> 2, items = 64 * r4;
  for (int o = 0; o < s.ops; ++o) {
    const int64_t slab = s.M * r;
    const int S = s.splits[o];
    for (int e = tid; e < items; e += 256) {
      const int t = e / r4, q = 4 * (e - t * r4);
      const float* part = s.part[o] + (t0 + t) * r + q;
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      if (ids[t] >= 0) {
        for (int z0 = 0; z0 < S; z0 += 8) {  // 8 slabs' loads in flight, summed in order
          f32x4 w[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (z0 + u < S) w[u] = *reinterpret_cast<const f32x4*>(part + (z0 + u) * slab);
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (z0 + u < S) x += w[u];
        }
        x *= sc[t];
      }
      const u32x2 h = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
      *reinterpret_cast<u32x2*>(&v[o][t * pitch + q]) = h;
      auto inf = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
      if (inf(h[0]) || inf(h[1])) spoilt[t] = 1;
      if (s.P[o] && t0 + t < s.M)
        *reinterpret_cast<u32x2*>(s.P[o] + (t0 + t) * r + q) = bad[t] ? u32x2{0x7FC07FC0u, 0x7FC07FC0u} : h;
    }
  }
  if (!s.Pt[0]) return;
  __syncthreads();
  if (tid < 64) {
    const int a = ids[tid];
    const uint64_t m = __ballot(a >= 0 && !spoilt[tid]);
    if (tid == 0) reinterpret_cast<uint64_t*>(s.mask)[blockIdx.x] = m;
    if (a >= 0 && spoilt[tid]) s.gbad[a] = 1;  // (more than one may store it)
  }
  const int64_t M8 = (s.M + 7) / 8 * 8;
  const int c = (tid & 7) * 8;  // this thread's 8 tokens
  int mine[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mine[k] = spoilt[c + k] ? -1 : ids[c + k];
  if (t0 + c >= M8) return;
  for (int i = 0; i < ngroups; ++i) {
    const int g = groups[i], rows = min(s.per, s.n - g * s.per) * r;
    for (int row = tid >> 3; row < rows; row += 32) {
      const int k0 = row / r, a = g * s.per + k0, q = row - k0 * r;
      for (int o = 0; o < s.ops; ++o) {
        uint32_t w[4];
        auto at = [&](int k) { return mine[k] == a ? (uint32_t)v[o][(c + k) * pitch + q] : 0u; };
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = at(2 * k) | at(2 * k + 1) << 16;
        *reinterpret_cast<u32x4*>(s.Pt[o] + ((int64_t)g * s.per * r + row) * M8 + t0 + c) = u32x4{w[0], w[1], w[2], w[3]};
      }
    }
  }
}

// Strips in fp32 by dot products, for few rows and for fp32: X and the rows of A come
// from the caches, so what bounds a few rows is the latency of a launch with two loads
// in a row (48 x 4096, r = 16: 6.8 us; 1 row 5.3).  blockIdx.z 0: P [M, r] = s_a X A_a^T, one wave a
// value, 16 bytes of both rows a lane; 1: Q [M, r] = s_a dY B_a with B [n][N, r] as
// it is, one wave 8 values, a lane an element of dY's row and 8 ranks of B's.
template <typename T>
__global__ void __launch_bounds__(256) multi_dot_kernel(const MultiDot d) {
  constexpr int E = 16 / sizeof(T);
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = blockIdx.y * 4 + (threadIdx.x >> 6);
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
    for (int i = threadIdx.x; i < d.nzero; i += 256) d.zero[i] = 0;
  const int a = adapter_at(d.index, t, d.M, d.n), r = d.r;
  if (blockIdx.z == 0) {
    const int q = wave;
    if (q >= r) return;
    float s = 0.f;
    if (a >= 0) {
      const u32x4* x = reinterpret_cast<const u32x4*>(static_cast<const T*>(d.X) + t * d.K);
      const u32x4* w = reinterpret_cast<const u32x4*>(static_cast<const T*>(d.A) + ((int64_t)a * r + q) * d.K);
#pragma unroll 8
      for (int64_t k = lane; k < d.K / E; k += 64) {
        const u32x4 u = x[k], v = w[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t ue = u[e], ve = v[e];  // (a vector's element has no address to cast at)
          if constexpr (sizeof(T) == 2) {
            s = __builtin_fmaf(__builtin_bit_cast(float, ue << 16), __builtin_bit_cast(float, ve << 16), s);
            s = __builtin_fmaf(__builtin_bit_cast(float, ue & 0xFFFF0000u), __builtin_bit_cast(float, ve & 0xFFFF0000u), s);
          } else {
            s = __builtin_fmaf(__builtin_bit_cast(float, ue), __builtin_bit_cast(float, ve), s);
          }
        }
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
      s *= d.scales[a];
    }
    if (lane == 0) d.P[t * r + q] = s;
    return;
  }
  const int q = 8 * wave;
  if (q >= r) return;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.f;
  if (a >= 0) {
    const T* g = static_cast<const T*>(d.dY) + t * d.N;
    const T* b = static_cast<const T*>(d.B) + (int64_t)a * d.N * r + q;
#pragma unroll 8
    for (int64_t k = lane; k < d.N; k += 64) {
      const float x = val(g[k]);
      const u32x4* w = reinterpret_cast<const u32x4*>(b + k * r);
#pragma unroll
      for (int h = 0; h < 8 / E; ++h) {
        const u32x4 v = w[h];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t u = v[e * sizeof(T) / 4];
          s[h * E + e] = __builtin_fmaf(x, __builtin_bit_cast(float, sizeof(T) == 4 ? u : e & 1 ? u & 0xFFFF0000u : u << 16), s[h * E + e]);
        }
      }
    }
  }
  const float sc = a >= 0 ? d.scales[a] : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[e] += __shfl_xor(s[e], o);
    if (lane == e) d.Q[t * r + q + e] = a >= 0 ? s[e] * sc : 0.f;
  }
}

// out [M, K] = Q_t A_a, A [n][r, K]: a thread 16 bytes of a row.
template <typename T>
__global__ void __launch_bounds__(256) multi_update_rows_kernel(const float* Q, const T* A, const int* index, int64_t M, int64_t K,
                                                                int n, int r, T* out) {
  constexpr int E = 16 / sizeof(T);
  const int64_t t = blockIdx.y, k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * E;
  if (k >= K) return;
  const int a = adapter_at(index, t, M, n);
  float s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = 0.f;
  if (a >= 0) {
    const T* w = A + (int64_t)a * r * K + k;
    const float* p = Q + t * r;
#pragma unroll 8
    for (int q = 0; q < r; ++q) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(w + (int64_t)q * K);
      const float x = p[q];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t u = v[e * sizeof(T) / 4];
        s[e] = __builtin_fmaf(x, __builtin_bit_cast(float, sizeof(T) == 4 ? u : e & 1 ? u & 0xFFFF0000u : u << 16), s[e]);
      }
    }
  }
  u32x4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 2)
      o[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
    else
      o[e] = __builtin_bit_cast(uint32_t, s[e]);
  }
  *reinterpret_cast<u32x4*>(out + t * K + k) = o;
}

// out [M, N] = P_t . B_a[j, :], B [n][N, r]; a thread one output, 16 bytes of B
// at a time.
template <typename T, typename TP>
__global__ void __launch_bounds__(256) multi_update_kernel(const TP* P, const T* B, const int* index, int64_t M, int64_t N,
                                                           int n, int r, T* out) {
  constexpr int E = 16 / sizeof(T);
  const int64_t t = blockIdx.y, j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= N) return;
  const int a = adapter_at(index, t, M, n);
  float s = 0.f;
  if (a >= 0) {
    const u32x4* b = reinterpret_cast<const u32x4*>(B + ((int64_t)a * N + j) * r);
    const TP* p = P + t * r;
#pragma unroll 4
    for (int q = 0; q < r / E; ++q) {
      const u32x4 v = b[q];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t u = v[e * sizeof(T) / 4];
        const float x = __builtin_bit_cast(float, sizeof(T) == 4 ? u : e & 1 ? u & 0xFFFF0000u : u << 16);
        s = __builtin_fmaf(val(p[q * E + e]), x, s);
      }
    }
  }
  store_out<T>(out, t * N + j, s);
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// bf16: partials of dB^T and dA for one row group each (gemm_panel.h), both in
// one launch: grid rows [0, s0) are the splits of the first.  64 rows of the stacked
// adapters a block: the adapters of one block share the tokens that it streams, and in
// a batch's order each 64-token tile is listed once or twice (8192 tokens, 4096 + 4096
// columns, 8 adapters of 16: 134 MB in 37 us; in random order every group reads all: 290).
// Four stages where two blocks a CU need not share the LDS, else two.
template <int BR, int NS>
__global__ void __launch_bounds__(sdma::NT) __attribute__((amdgpu_waves_per_eu(1, 2)))
multi_grad_kernel(const GemmPair q, int s1, int rows, int total) {
  const int y = (int)blockIdx.y, w = y >= q.s0 ? 1 : 0, g = blockIdx.z;
  if ((int64_t)blockIdx.x * sdma::BN >= q.g[w].n_store) return;
  GemmArgs p = q.g[w];
  p.a1 = static_cast<const uint16_t*>(p.a1) + (int64_t)g * rows * p.lda1;
  p.c = static_cast<float*>(p.c) + (int64_t)g * rows * p.ldc;
  p.m_load = p.m_store = min(rows, total - g * rows);
  __shared__ __attribute__((aligned(1024))) char smem[sdma::Cfg<BR, NS>::LDS];
  splitnn_dma_tile<BR, NS, true>(smem, p, (int)blockIdx.x, w ? y - q.s0 : y, g, w ? s1 : q.s0);
}

// out [n r, N] = the sum over splits of part [splits][n r, N]; transposed within
// each adapter, [n][N, r], where tr.  Two of them in one launch (8 adapters of 16 over
// 4096 + 4096, 4 splits: 8 us).
template <typename T>
__global__ void __launch_bounds__(256) multi_grad_sum_kernel(const MultiGradSum g0, const MultiGradSum g1, const int* gbad, int n, int r) {
  const int w = (int)blockIdx.z >= n ? 1 : 0;
  const MultiGradSum& g = w ? g1 : g0;
  const int64_t a = (int64_t)blockIdx.z - (w ? n : 0);
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  if (c0 >= g.N) return;
  __shared__ float tile[64][33];
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int64_t stride = (int64_t)n * r * g.N;
  const float spoil = gbad && gbad[a] ? __builtin_nanf("") : 0.f;
  for (int q0 = 0; q0 < r; q0 += 32) {
    const int rows = min(32, r - q0);
    if (g.tr) __syncthreads();
    for (int k = y; k < rows; k += 4) {
      const int64_t at = (a * r + q0 + k) * g.N + c0 + x;
      float s = 0.f;
      if (c0 + x < g.N)
        for (int z = 0; z < g.splits; ++z) s += g.part[z * stride + at];
      s += spoil;
      if (g.tr)
        tile[x][k] = s;
      else if (c0 + x < g.N)
        store_out<T>(g.out, at, s);
    }
    if (!g.tr) continue;
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * rows; e += 256) {
      const int c = e / rows, k = e - c * rows;
      if (c0 + c < g.N) store_out<T>(g.out, (a * g.N + c0 + c) * r + q0 + k, tile[c][k]);
    }
  }
}

// Simple gradients, from fp32 strips: out [n][r, N] (or [n][N, r], tr) = sum over the
// adapter's tokens of P[t, q] X[t, j].  A block is 64 columns of one adapter over a
// range of tokens (partials [splits][n r, N] where there are several), a wave a
// quarter of the ranks, QK at most; tokens in order, 64 at a time: the adapter's
// are found, their strips go to LDS, 8 rows of X are in flight.  Every block looks
// through all indexes of its range: few rows only (128 rows, 256 + 256 columns, 4 adapters
// of 8: 10 us).
template <typename T, typename TO, int QK>
__global__ void __launch_bounds__(256) multi_outer_kernel(const MultiOuter o0, const MultiOuter o1, const int* index, int64_t M, int n, int r,
                                                          int splits) {
  const int w = (int)blockIdx.z >= splits ? 1 : 0;
  const MultiOuter& o = w ? o1 : o0;
  const int z = blockIdx.z - (w ? splits : 0);
  const int64_t j = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  if ((int64_t)blockIdx.x * 64 >= o.N) return;
  __shared__ int list[64];
  __shared__ int found;
  __shared__ __attribute__((aligned(16))) float strip[64][4 * QK];
  const int a = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* X = static_cast<const T*>(o.X);
  const int64_t per = ((M + splits - 1) / splits + 63) / 64 * 64, end = min(M, (z + 1) * per);
  float acc[QK];
#pragma unroll
  for (int k = 0; k < QK; ++k) acc[k] = 0.f;
  for (int64_t t0 = z * per; t0 < end; t0 += 64) {
    __syncthreads();
    if (wave == 0) {
      const bool is = adapter_at(index, t0 + lane, end, n) == a;
      const uint64_t m = __ballot(is);
      if (is) list[__popcll(m & ((1ull << lane) - 1))] = lane;
      if (lane == 0) found = __popcll(m);
    }
    __syncthreads();
    const int cnt = found;
    if (cnt == 0) continue;  // (uniform)
    for (int e = threadIdx.x; e < cnt * 4 * QK; e += 256) {
      const int i = e / (4 * QK), q = e - i * 4 * QK;
      strip[i][q] = q < r ? o.P[(t0 + list[i]) * r + q] : 0.f;
    }
    __syncthreads();
    for (int i0 = 0; i0 < cnt; i0 += 8) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i0 + u < cnt && j < o.N ? val(X[(t0 + list[i0 + u]) * o.N + j]) : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u < cnt) {
#pragma unroll
          for (int k = 0; k < QK; ++k) acc[k] = __builtin_fmaf(strip[i0 + u][wave * QK + k], x[u], acc[k]);
        }
    }
  }
  if (j >= o.N) return;
#pragma unroll
  for (int k = 0; k < QK; ++k) {
    const int q = wave * QK + k;
    if (q >= r) continue;
    const int64_t at = ((int64_t)a * r + q) * o.N + j;
    if (splits > 1)
      o.part[(int64_t)z * n * r * o.N + at] = acc[k];
    else
      store_out<TO>(o.out, o.tr ? ((int64_t)a * o.N + j) * r + q : at, acc[k]);
  }
}

}  // namespace

hipError_t launch_multi_lists(MultiLists q, hipStream_t st) {
  auto tiles = [&](const MultiTranspose& t) { return t.src ? (t.R + 31) / 32 * ((t.C + 63) / 64) * q.n : 0; };
  q.tr0 = tiles(q.tr[0]);
  const int64_t blocks = (int64_t)q.t128 + q.t256 + q.groups + (int64_t)q.n * q.chunks + q.tr0 + tiles(q.tr[1]);
  for (const MultiTranspose& t : q.tr)
    if (t.src && (t.R % 8 || t.C % 8)) return hipErrorInvalidValue;
  if (blocks <= 0) return hipSuccess;
  if (q.M <= 0 || q.n < 1 || blocks > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL(multi_lists_kernel, dim3((unsigned)blocks), dim3(256), 0, st, q);
  return hipGetLastError();
}

static bool panel_ok(const GemmArgs& a) {
  return a.ad_r >= 8 && a.ad_r <= kMultiMaxRank && a.ad_r % 8 == 0 && a.K1 % 8 == 0 && a.m_load == a.m_store &&
         panel_dma_fits(64, a.lda1, a.ldb1);
}

hipError_t launch_multi_panel(const GemmArgs& a, int sa, const GemmArgs* b, int sb, hipStream_t st) {
  if (a.m_store <= 0) return hipSuccess;
  const int64_t tiles = (a.m_store + PANEL_BM - 1) / PANEL_BM, cols = ((int64_t)a.ad_cap * a.ad_r + 63) / 64;
  if (!panel_ok(a) || sa < 1 || tiles > INT32_MAX || sa + sb > 65535 ||
      (b && (!panel_ok(*b) || sb < 1 || b->m_store != a.m_store || b->ad_cap != a.ad_cap || b->ad_r != a.ad_r)))
    return hipErrorInvalidValue;
  const GemmPair q{{a, b ? *b : a}, sa};
  const int64_t y = sa + (b ? sb : 0), z = std::max<int64_t>(1, std::min<int64_t>(cols, 384 / (tiles * y)));
  hipLaunchKernelGGL(multi_panel_kernel, dim3((unsigned)tiles, (unsigned)y, (unsigned)z), dim3(pdma::NT),
                     0, st, q);
  return hipGetLastError();
}

hipError_t launch_multi_strip(const MultiStrip& s, hipStream_t st) {
  if (s.M <= 0) return hipSuccess;
  if (s.r < 1 || s.r > kMultiMaxRank || s.M > INT32_MAX || s.ops < 1 || s.ops > 2) return hipErrorInvalidValue;
  hipLaunchKernelGGL(multi_strip_kernel, dim3((unsigned)((s.M + 63) / 64)), dim3(256), 0, st, s);
  return hipGetLastError();
}

hipError_t launch_multi_gemm(GemmArgs a, bool low, hipStream_t st) {
  const int bm = low ? w4h::BM : w4::BM;
  const int64_t ld = std::max<int64_t>(a.lda1, std::max<int64_t>(a.ldb1, a.ad_r));
  const int64_t tm = (a.m_store + bm - 1) / bm, tn = (a.n_store + w4::BN - 1) / w4::BN;
  if (a.m_load != a.m_store || a.n_load != a.n_store || a.n_store % 8 || a.K1 < w4::BK || a.K1 % 8 ||
      !whole_ld_fits(std::max(ld, a.ldc)) || tm * tn > INT32_MAX || a.ad_r < 8 || a.ad_r % 8 || a.lda2 != a.ad_r ||
      a.ad_cap > bm)
    return hipErrorInvalidValue;
  if (tm * tn == 0) return hipSuccess;
  a.tiles_m = (int)tm;
  if (low) {
    hipLaunchKernelGGL((gemm_w4_half_kernel<EPI_ACT, true>), dim3((unsigned)(tm * tn)), dim3(w4::NT), 0, st, a);
    return hipGetLastError();
  }
  if (a.st_full < 0 || a.st_half < 0 || a.st_full + (int64_t)a.st_half != tm * tn ||
      a.st_full + 2 * (int64_t)a.st_half > INT32_MAX ||
      (a.st_half > 0 && (!a.st_part || !a.st_cnt || a.st_early < 0 || a.K1 / w4::BK / 2 - a.st_early < 2)))
    return hipErrorInvalidValue;
  // whole tiles store from the accumulators, without the passes through LDS that
  // ragged ones need (8192 x 4096 over 4096: 205 against 219 us)
  if (a.st_half == 0 && a.m_store % w4::BM == 0 && a.n_store % w4::BN == 0)
    hipLaunchKernelGGL((gemm_w4_stream_kernel<EPI_STORE, true>), dim3((unsigned)a.st_full), dim3(w4::NT), 0, st, a);
  else
    hipLaunchKernelGGL((gemm_w4_stream_kernel<EPI_ACT, true>), dim3((unsigned)(a.st_full + 2 * a.st_half)), dim3(w4::NT), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_multi_dot(int elem_bytes, const MultiDot& d, hipStream_t st) {
  if (d.M <= 0) return hipSuccess;
  if (d.M > INT32_MAX || d.r % 8 || d.K % 8) return hipErrorInvalidValue;
  const dim3 grid((unsigned)d.M, (unsigned)((d.r + 3) / 4), d.Q ? 2u : 1u);
  if (elem_bytes == 2)
    hipLaunchKernelGGL((multi_dot_kernel<uint16_t>), grid, dim3(256), 0, st, d);
  else
    hipLaunchKernelGGL((multi_dot_kernel<float>), grid, dim3(256), 0, st, d);
  return hipGetLastError();
}

hipError_t launch_multi_update_rows(int elem_bytes, const float* Q, const void* A, const int* index, int64_t M, int64_t K, int n, int r,
                                    void* out, hipStream_t st) {
  if (K % 8) return hipErrorInvalidValue;
  for (int64_t t0 = 0; t0 < M; t0 += 65535) {  // (rows on the grid's y)
    const int64_t m = std::min<int64_t>(65535, M - t0);
    const dim3 grid((unsigned)((K * elem_bytes / 16 + 255) / 256), (unsigned)m);
    if (elem_bytes == 2)
      hipLaunchKernelGGL((multi_update_rows_kernel<uint16_t>), grid, dim3(256), 0, st, Q + t0 * r, static_cast<const uint16_t*>(A),
                         index + t0, m, K, n, r, static_cast<uint16_t*>(out) + t0 * K);
    else
      hipLaunchKernelGGL((multi_update_rows_kernel<float>), grid, dim3(256), 0, st, Q + t0 * r, static_cast<const float*>(A), index + t0,
                         m, K, n, r, static_cast<float*>(out) + t0 * K);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_multi_update(int elem_bytes, const void* P, bool P32, const void* B, const int* index, int64_t M, int64_t N,
                               int n, int r, void* out, hipStream_t st) {
  if (elem_bytes == 4 && !P32) return hipErrorInvalidValue;
  // (rows on the grid's y, 65535 at most)
  for (int64_t t0 = 0; t0 < M; t0 += 65535) {
    const int64_t m = std::min<int64_t>(65535, M - t0);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)m);
    const float* p32 = static_cast<const float*>(P) + t0 * r;
    const uint16_t* p16 = static_cast<const uint16_t*>(P) + t0 * r;
    if (elem_bytes == 4)
      hipLaunchKernelGGL((multi_update_kernel<float, float>), grid, dim3(256), 0, st, p32, static_cast<const float*>(B), index + t0,
                         m, N, n, r, static_cast<float*>(out) + t0 * N);
    else if (P32)
      hipLaunchKernelGGL((multi_update_kernel<uint16_t, float>), grid, dim3(256), 0, st, p32, static_cast<const uint16_t*>(B),
                         index + t0, m, N, n, r, static_cast<uint16_t*>(out) + t0 * N);
    else
      hipLaunchKernelGGL((multi_update_kernel<uint16_t, uint16_t>), grid, dim3(256), 0, st, p16, static_cast<const uint16_t*>(B),
                         index + t0, m, N, n, r, static_cast<uint16_t*>(out) + t0 * N);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_multi_grad(const GemmArgs& a, int sa, const GemmArgs& b, int sb, int rows, int total, hipStream_t st) {
  auto ok = [&](const GemmArgs& g) {
    return g.n_load == g.n_store && g.n_store % 8 == 0 && g.n_store > 0 && sdma::BK * g.ldb1 * 2 + g.n_store * 2 < (int64_t)w4::BIG &&
           g.lda1 * 2 * 128 < (int64_t)w4::BIG;
  };
  const int64_t groups = (total + rows - 1) / rows;
  if (rows < 1 || rows > 128 || total < 1 || sa < 1 || sb < 1 || sa + sb > 65535 || groups > 65535 || !ok(a) || !ok(b))
    return hipErrorInvalidValue;
  const GemmPair q{{a, b}, sa};
  const int64_t t = (std::max(a.n_store, b.n_store) + sdma::BN - 1) / sdma::BN;
  const dim3 grid((unsigned)t, (unsigned)(sa + sb), (unsigned)groups);
  if (rows <= 64 && t * (sa + sb) * groups <= 512)
    hipLaunchKernelGGL((multi_grad_kernel<64, 4>), grid, dim3(sdma::NT), 0, st, q, sb, rows, total);
  else if (rows <= 64)
    hipLaunchKernelGGL((multi_grad_kernel<64, 2>), grid, dim3(sdma::NT), 0, st, q, sb, rows, total);
  else
    hipLaunchKernelGGL((multi_grad_kernel<128, 3>), grid, dim3(sdma::NT), 0, st, q, sb, rows, total);
  return hipGetLastError();
}

hipError_t launch_multi_grad_sum(int out_bytes, const MultiGradSum& a, const MultiGradSum& b, const int* gbad, int n, int r,
                                 hipStream_t st) {
  if (n < 1 || 2 * (int64_t)n > 65535) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((std::max(a.N, b.N) + 63) / 64), 1, (unsigned)(2 * n));
  if (out_bytes == 2)
    hipLaunchKernelGGL((multi_grad_sum_kernel<uint16_t>), grid, dim3(256), 0, st, a, b, gbad, n, r);
  else
    hipLaunchKernelGGL((multi_grad_sum_kernel<float>), grid, dim3(256), 0, st, a, b, gbad, n, r);
  return hipGetLastError();
}

namespace {
template <typename T, typename TO>
void run_outer(const MultiOuter& a, const MultiOuter& b, const int* index, int64_t M, int n, int r, int splits, hipStream_t st) {
  const dim3 grid((unsigned)((std::max(a.N, b.N) + 63) / 64), (unsigned)n, (unsigned)(2 * splits));
  auto go = [&](auto qk) {
    hipLaunchKernelGGL((multi_outer_kernel<T, TO, decltype(qk)::value>), grid, dim3(256), 0, st, a, b, index, M, n, r, splits);
  };
  if (r <= 8)
    go(std::integral_constant<int, 2>{});
  else if (r <= 16)
    go(std::integral_constant<int, 4>{});
  else if (r <= 32)
    go(std::integral_constant<int, 8>{});
  else if (r <= 64)
    go(std::integral_constant<int, 16>{});
  else
    go(std::integral_constant<int, 32>{});
}
}  // namespace

hipError_t launch_multi_outer(int elem_bytes, const MultiOuter& a, const MultiOuter& b, const int* index, int64_t M, int n, int r, int splits,
                              int out_bytes, hipStream_t st) {
  if (M < 1 || n < 1 || n > 65535 || r > kMultiMaxRank || splits < 1 || splits > 32 || (splits > 1 && (!a.part || !b.part)))
    return hipErrorInvalidValue;
  if (elem_bytes == 2)
    out_bytes == 2 ? run_outer<uint16_t, uint16_t>(a, b, index, M, n, r, splits, st)
                   : run_outer<uint16_t, float>(a, b, index, M, n, r, splits, st);
  else
    out_bytes == 2 ? run_outer<float, uint16_t>(a, b, index, M, n, r, splits, st) : run_outer<float, float>(a, b, index, M, n, r, splits, st);
  return hipGetLastError();
}

}  // namespace lora
