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

constexpr int kScanPieces = 4096;  // 16-byte pieces of a block that looks for infinities

__device__ __forceinline__ int adapter_at(const int* index, int64_t t, int64_t M, int n) {
  const int a = t < M ? index[t] : -1;
  return a >= 0 && a < n ? a : -1;
}

// ---------------------------------------------------------------------------
// lists.  Blocks [0, T128): the adapters of a 128-row tile, in the order of
// their first rows; then T256 blocks, of a 256-row tile; then the row groups of
// the gradients: the 64-token tiles in which an adapter of the group occurs.
// The first block also clears the stream kernel's counters.  Then `chunks` blocks
// an adapter, which look for infinities and NaNs in their 64 KB of its second
// operand if a row carries it: one adapter's must not reach the others' rows.
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

__global__ void __launch_bounds__(256) multi_lists_kernel(const MultiLists q) {
  __shared__ int ids[256];
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
    const int64_t end = min((int64_t)(c + 1) * kScanPieces, q.scan16);
    const u32x4* v = reinterpret_cast<const u32x4*>(q.scan) + (int64_t)a * q.scan16;
    uint32_t found = 0;
#pragma unroll 8
    for (int64_t i = (int64_t)c * kScanPieces + tid; i < end; i += 256) {
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
// bf16: partials of the tile's strips (gemm_panel.h), column groups of 64 past
// the tile's own leave at once.  Two of them in one launch (the backward's P
// and Q): splits [0, s0) of the grid are the first one's.
__global__ void __launch_bounds__(pdma::NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
multi_panel_kernel(const GemmPair q) {
  const int y = (int)blockIdx.z, w = y >= q.s0 ? 1 : 0;
  __shared__ __attribute__((aligned(1024))) char smem[pdma::Cfg<PANEL_BM, 64>::LDS];
  const GemmArgs& p = q.g[w];
  const int mt = blockIdx.x, cg = blockIdx.y;
  if (64 * cg >= scalar_at(p.ad_cnt, mt) * p.ad_r) return;
  panel_dma_tile<PANEL_BM, 64, true>(smem, p, mt, w ? y - q.s0 : y, cg);
}

// The strips of a 64-token tile from their partials, bf16(s_a sum), of one or
// both operands: `P` [M, r] for the product (NaNs for a row whose adapter's
// second operand is spoilt, which its tiles' lists are told here), and, for the
// gradients, `Pt` [n r, M8]: the strips spread over their group's rows, zeros
// where a token has another adapter, for the groups that the tile meets.  A token
// with an infinity or NaN in a strip (its own row of X or dY has one then) would
// reach the other adapters of its group as zero times that: its strips are zeros
// there, its bit in `mask` is clear like that of a token without adapter, and
// its adapter's gradients are NaNs (gbad).
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

// fp32 strips P [M, r], one wave a value; rows of whole 16-byte pieces.
template <typename T>
__global__ void __launch_bounds__(256) multi_dot_kernel(const T* X, const T* A, const float* scales, const int* index,
                                                        int64_t M, int64_t K, int n, int r, float* P, int* zero, int nzero) {
  constexpr int E = 16 / sizeof(T);
  const int64_t t = blockIdx.x;
  const int q = blockIdx.y * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < nzero; i += 256) zero[i] = 0;
  if (q >= r) return;
  const int a = adapter_at(index, t, M, n);
  float s = 0.f;
  if (a >= 0) {
    const u32x4* x = reinterpret_cast<const u32x4*>(X + t * K);
    const u32x4* w = reinterpret_cast<const u32x4*>(A + ((int64_t)a * r + q) * K);
#pragma unroll 8
    for (int64_t k = lane; k < K / E; k += 64) {
      const u32x4 u = x[k], v = w[k];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) {
          s = __builtin_fmaf(__builtin_bit_cast(float, u[e] << 16), __builtin_bit_cast(float, v[e] << 16), s);
          s = __builtin_fmaf(__builtin_bit_cast(float, u[e] & 0xFFFF0000u), __builtin_bit_cast(float, v[e] & 0xFFFF0000u), s);
        } else {
          const uint32_t ue = u[e], ve = v[e];  // (a vector's element has no address to cast at)
          s = __builtin_fmaf(__builtin_bit_cast(float, ue), __builtin_bit_cast(float, ve), s);
        }
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    s *= scales[a];
  }
  if (lane == 0) P[t * r + q] = s;
}

// out [M, N] (+)= P_t . B_a[j, :], B [n][N, r]; a thread one output, 16 bytes of B
// at a time.
template <typename T, typename TP>
__global__ void __launch_bounds__(256) multi_update_kernel(const TP* P, const T* B, const int* index, int64_t M, int64_t N,
                                                           int n, int r, int add, T* out) {
  constexpr int E = 16 / sizeof(T);
  const int64_t t = blockIdx.y, j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= N) return;
  const int a = adapter_at(index, t, M, n);
  float s = add ? val(out[t * N + j]) : 0.f;
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

// dst [n][C, R] = src [n][R, C] transposed, through 32 x 32 tiles; two stacks in
// one launch (blockIdx.z < n: the first).
template <typename T>
__global__ void __launch_bounds__(256) multi_transpose_kernel(const MultiTranspose a, const MultiTranspose b, int n) {
  __shared__ T tile[32][33];
  const int w = (int)blockIdx.z >= n ? 1 : 0;
  const MultiTranspose& q = w ? b : a;
  const int64_t z = (int64_t)blockIdx.z - (w ? n : 0);
  const int64_t tc = (q.C + 31) / 32, id = blockIdx.x;
  if (id >= tc * ((q.R + 31) / 32)) return;
  const int64_t r0 = id / tc * 32, c0 = id % tc * 32;
  const T* src = static_cast<const T*>(q.src) + z * q.R * q.C;
  T* dst = static_cast<T*>(q.dst) + z * q.R * q.C;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int k = y; k < 32; k += 8)
    if (r0 + k < q.R && c0 + x < q.C) tile[k][x] = src[(r0 + k) * q.C + c0 + x];
  __syncthreads();
  for (int k = y; k < 32; k += 8)
    if (c0 + k < q.C && r0 + x < q.R) dst[(c0 + k) * q.R + r0 + x] = tile[x][k];
}

// ---------------------------------------------------------------------------
// gradients
// ---------------------------------------------------------------------------
// bf16: partials of dB^T and dA for one row group each (gemm_panel.h), both in
// one launch: grid rows [0, s0) are the splits of the first.
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
// each adapter, [n][N, r], where tr.  Two of them in one launch.
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
  const float spoil = gbad[a] ? __builtin_nanf("") : 0.f;
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

// fp32: out [n][r, N] (or [n][N, r], tr) = sum over the adapter's tokens of
// P[t, q] X[t, j]; a block is 64 columns and one adapter, a thread one column
// and a quarter of the ranks; tokens in order.
template <typename T, typename TO>
__global__ void __launch_bounds__(256) multi_outer_kernel(const float* P, const T* X, const int* index, int64_t M, int64_t N,
                                                          int n, int r, int tr, TO* out) {
  __shared__ int ids[256];
  const int a = blockIdx.y, x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int64_t j = (int64_t)blockIdx.x * 64 + x;
  float acc[32];
#pragma unroll
  for (int k = 0; k < 32; ++k) acc[k] = 0.f;
  for (int64_t t0 = 0; t0 < M; t0 += 256) {
    __syncthreads();
    ids[threadIdx.x] = adapter_at(index, t0 + threadIdx.x, M, n);
    __syncthreads();
    for (int i = 0; i < 256; ++i) {
      if (ids[i] != a) continue;
      const float v = j < N ? val(X[(t0 + i) * N + j]) : 0.f;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (y + 4 * k < r) acc[k] = __builtin_fmaf(P[(t0 + i) * r + y + 4 * k], v, acc[k]);
    }
  }
  if (j >= N) return;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const int q = y + 4 * k;
    if (q < r) store_out<TO>(out, tr ? ((int64_t)a * N + j) * r + q : ((int64_t)a * r + q) * N + j, acc[k]);
  }
}

}  // namespace

hipError_t launch_multi_lists(const MultiLists& q, hipStream_t st) {
  const int64_t blocks = (int64_t)q.t128 + q.t256 + q.groups + (int64_t)q.n * q.chunks;
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
  if (!panel_ok(a) || sa < 1 || tiles > INT32_MAX || cols > 65535 ||
      (b && (!panel_ok(*b) || sb < 1 || b->m_store != a.m_store || b->ad_cap != a.ad_cap || b->ad_r != a.ad_r)))
    return hipErrorInvalidValue;
  const GemmPair q{{a, b ? *b : a}, sa};
  hipLaunchKernelGGL(multi_panel_kernel, dim3((unsigned)tiles, (unsigned)cols, (unsigned)(sa + (b ? sb : 0))), dim3(pdma::NT),
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
  hipLaunchKernelGGL((gemm_w4_stream_kernel<EPI_ACT, true>), dim3((unsigned)(a.st_full + 2 * a.st_half)), dim3(w4::NT), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_multi_dot(int elem_bytes, const void* X, const void* A, const float* scales, const int* index, int64_t M,
                            int64_t K, int n, int r, float* P, hipStream_t st, int* zero, int nzero) {
  if (M <= 0) return hipSuccess;
  if (M > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)M, (unsigned)((r + 3) / 4));
  if (elem_bytes == 2)
    hipLaunchKernelGGL((multi_dot_kernel<uint16_t>), grid, dim3(256), 0, st, static_cast<const uint16_t*>(X),
                       static_cast<const uint16_t*>(A), scales, index, M, K, n, r, P, zero, nzero);
  else
    hipLaunchKernelGGL((multi_dot_kernel<float>), grid, dim3(256), 0, st, static_cast<const float*>(X),
                       static_cast<const float*>(A), scales, index, M, K, n, r, P, zero, nzero);
  return hipGetLastError();
}

hipError_t launch_multi_update(int elem_bytes, const void* P, bool P32, const void* B, const int* index, int64_t M, int64_t N,
                               int n, int r, bool add, void* out, hipStream_t st) {
  if (elem_bytes == 4 && !P32) return hipErrorInvalidValue;
  // (rows on the grid's y, 65535 at most)
  for (int64_t t0 = 0; t0 < M; t0 += 65535) {
    const int64_t m = std::min<int64_t>(65535, M - t0);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)m);
    const float* p32 = static_cast<const float*>(P) + t0 * r;
    const uint16_t* p16 = static_cast<const uint16_t*>(P) + t0 * r;
    if (elem_bytes == 4)
      hipLaunchKernelGGL((multi_update_kernel<float, float>), grid, dim3(256), 0, st, p32, static_cast<const float*>(B), index + t0,
                         m, N, n, r, add ? 1 : 0, static_cast<float*>(out) + t0 * N);
    else if (P32)
      hipLaunchKernelGGL((multi_update_kernel<uint16_t, float>), grid, dim3(256), 0, st, p32, static_cast<const uint16_t*>(B),
                         index + t0, m, N, n, r, add ? 1 : 0, static_cast<uint16_t*>(out) + t0 * N);
    else
      hipLaunchKernelGGL((multi_update_kernel<uint16_t, uint16_t>), grid, dim3(256), 0, st, p16, static_cast<const uint16_t*>(B),
                         index + t0, m, N, n, r, add ? 1 : 0, static_cast<uint16_t*>(out) + t0 * N);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_multi_transpose(int elem_bytes, const MultiTranspose& a, const MultiTranspose* b, int n, hipStream_t st) {
  auto tiles = [](const MultiTranspose& q) { return (q.R + 31) / 32 * ((q.C + 31) / 32); };
  const int64_t t = std::max(tiles(a), b ? tiles(*b) : 0);
  if (n < 1 || 2 * (int64_t)n > 65535 || t > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)t, 1, (unsigned)(b ? 2 * n : n));
  if (elem_bytes == 2)
    hipLaunchKernelGGL((multi_transpose_kernel<uint16_t>), grid, dim3(256), 0, st, a, b ? *b : a, n);
  else
    hipLaunchKernelGGL((multi_transpose_kernel<float>), grid, dim3(256), 0, st, a, b ? *b : a, n);
  return hipGetLastError();
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
  if (rows <= 64)
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

hipError_t launch_multi_outer(const float* P, const float* X, const int* index, int64_t M, int64_t N, int n, int r, bool tr,
                              int out_bytes, void* out, hipStream_t st) {
  if (n < 1 || n > 65535 || r > kMultiMaxRank) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)n);
  if (out_bytes == 2)
    hipLaunchKernelGGL((multi_outer_kernel<float, uint16_t>), grid, dim3(256), 0, st, P, X, index, M, N, n, r, tr ? 1 : 0,
                       static_cast<uint16_t*>(out));
  else
    hipLaunchKernelGGL((multi_outer_kernel<float, float>), grid, dim3(256), 0, st, P, X, index, M, N, n, r, tr ? 1 : 0,
                       static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace lora
