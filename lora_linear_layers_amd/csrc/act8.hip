// act8.hip - the two products of a LoRA backward that read the layer's input,
// with that input kept in 8 bits (norm.hip: e4m3 codes and a power of two a row):
//
//     P = s X A^T,   dA = Q^T X,   Q = s dY B,   X = diag(2^e) K
//
// A row's scale leaves both contractions: it multiplies P's row, and Q's row
// before the contraction over tokens.  What remains is K, whose values are bf16
// numbers, so the codes go to LDS as they are (DMA, half of bf16's bytes) and are
// expanded on the way from LDS to the matrix cores, four conversions a fragment of
// eight.  Nothing of X in bf16 is ever in memory.
//
// Both kernels are the layer's (gemm_panel.h), which are streams of X, with
// half of the bytes a stage and more stages in flight.  The panel's stage is 128
// elements deep, so that a row's piece stays 128 bytes (its A operand then has
// two 64-deep tiles a stage).  The gradient's fragments, eight tokens of a column,
// come through ds_read_b64_tr_b8: in each 16-lane group lane i points at 8 bytes of
// token row i / 2 and receives the group's 16 columns' byte i of eight rows.  Its LDS rows
// (64 tokens of 256 bytes) hold 16-byte chunk c at chunk c ^ 2 (row & 7): the
// eight rows of a group, two chunks each of two groups, then cover all 64 banks.
//
// 8192 tokens, 14336 -> 4096, r = 64, each in one launch with the bf16 half of the pair
// (dY B, dY^T P: 67 MB): codes and that, 185 MB, in 54 us both; a copy of X in bf16 and
// the layer's own kernels over it took 111 us more (unpacking 352 MB, reading 235 twice).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_panel.h"
#include "launch.h"

namespace lora {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// eight e4m3 codes as bf16 (exact)
__device__ __forceinline__ bf16x8 expand8(u32x2 v) {
  const uint32_t lo = v[0], hi = v[1];
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

namespace p8 {
constexpr int BM = PANEL_BM, BK = 128;
template <int BN>
struct Cfg {
  static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;  // B: two 64-deep tiles of B_BYTES
  static constexpr int STAGE = A_BYTES + 2 * B_BYTES;
  static constexpr int NS = 160 * 1024 / STAGE;
  static constexpr int IA = BM / 8 / 4, IB = BN / 8 / 4;
  static constexpr int PER = IA + 2 * IB;
  static constexpr int FM = BM / 2 / 32, FN = BN / 2 / 32;
  static constexpr int LDS = NS * STAGE;
  static_assert(IA % 2 == 0 && IB % 2 == 0 && NS >= 3, "row parity pattern of the DMA lane mapping; stages");
};
}  // namespace p8

// row tile mt over split z, as panel_dma_tile
template <int BN>
__device__ __forceinline__ void panel8_tile(char* smem, const Act8Args& p, const int mt, const int z) {
  using namespace p8;
  using C = Cfg<BN>;
  constexpr int NS = C::NS, LEAD = NS - 1, FM = C::FM, FN = C::FN;
  asm volatile("" ::: "a0");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, hh = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (int64_t)mt * BM;
  const int64_t kbeg = (int64_t)z * p.ksplit;
  const int64_t kend = kbeg + p.ksplit < p.d ? kbeg + p.ksplit : p.d;
  const int klen = kend > kbeg ? (int)(kend - kbeg) : 0;
  const int nk = (klen + BK - 1) / BK;

  const int dr = lane >> 3;
  const int dce = (lane & 7) ^ (lane >> 4), dco = (lane & 7) ^ ((lane >> 4) | 4);
  const char* ga = reinterpret_cast<const char*>(p.codes) + m0 * p.d + kbeg;
  const char* gb = reinterpret_cast<const char*>(p.A) + kbeg * 2;
  const int64_t mrem = p.M - m0;
  auto dma = [&](const char* base, char* dst, bool ok, uint32_t off) {
    uint32_t vo = ok ? off : w4::OOB;
    asm volatile("" : "+v"(vo));
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, w4::BIG, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, (int)vo, 0, 0, 0);
  };
  auto issue = [&](int u) {
    char* st = smem + (u % NS) * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::IA; ++i) {
      const int row = 8 * (i + C::IA * wave) + dr, kk = u * BK + 16 * (i & 1 ? dco : dce);
      dma(ga, st + 8 * (i + C::IA * wave) * 128, kk < klen && row < mrem, (uint32_t)(row * p.d + kk));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < C::IB; ++i) {
        const int row = 8 * (i + C::IB * wave) + dr, kk = u * BK + 64 * h + 8 * (i & 1 ? dco : dce);
        dma(gb, st + C::A_BYTES + h * C::B_BYTES + 8 * (i + C::IB * wave) * 128, kk < klen && row < p.r,
            (uint32_t)((row * p.d + kk) * 2));
      }
  };

  const int swz = (l32 >> 1) & 7;
  const uint32_t ra = (uint32_t)(wm * (BM / 2) + l32) * 128 + 8 * hh;
  const uint32_t rb = (uint32_t)C::A_BYTES + (uint32_t)(wn * (BN / 2) + l32) * 128;
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  if (nk > 0) {
#pragma unroll
    for (int u = 0; u < LEAD; ++u) issue(u);
    for (int t = 0; t < nk; ++t) {
      __builtin_amdgcn_s_waitcnt(pdma::vmcnt_imm(C::PER * (LEAD - 1)));
      lds_barrier();
      issue(t + LEAD);  // into stage t-1's slot; zeros past the end
      const char* st = smem + (t % NS) * C::STAGE;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        bf16x8 fa[FM], fb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[i] = expand8(*reinterpret_cast<const u32x2*>(st + ra + ((s ^ swz) << 4) + i * 32 * 128));
#pragma unroll
        for (int j = 0; j < FN; ++j)
          fb[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + rb + (s >> 2) * C::B_BYTES +
                                                                             ((((2 * s + hh) & 7) ^ swz) << 4) + j * 32 * 128));
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
      }
    }
    __builtin_amdgcn_s_waitcnt(pdma::vmcnt_imm(0));  // (as panel_dma_tile)
  }
  float* out = p.part + (int64_t)z * p.rows * p.r8;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int64_t row = m0 + wm * (BM / 2) + 32 * i + 8 * (v >> 2) + 4 * hh + (v & 3);
      if (row >= p.rows) continue;
      const float sc = row < p.M ? p.scale8[row] : 0.f;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int col = wn * (BN / 2) + 32 * j + l32;
        if (col < p.r8) out[row * p.r8 + col] = acc[i][j][v] * sc;
      }
    }
}

namespace s8 {
constexpr int BN = 256, BK = 64, B_BYTES = BK * BN;
template <int BR, int NS_>
struct Cfg {
  static constexpr int A_BYTES = BR * 128, STAGE = A_BYTES + B_BYTES, NS = NS_;
  static constexpr int IA = BR / 8 / 4, IB = BK / 4 / 4, PER = IA + IB;
  static constexpr int FM = BR / 32, FN = 2;
  static constexpr int LDS = NS * STAGE;
  static_assert(IA % 2 == 0 && NS >= 3 && LDS <= 160 * 1024, "row parity pattern; stages; the ring fits the LDS");
};

// the four steps' fragments of a stage, 8 codes each: reads at a, and a + 4096 a step
template <int FN>
__device__ __forceinline__ void tr_codes(u32x2 (&f)[4][FN], const uint32_t (&a)[FN]) {
  static_assert(FN == 2, "two column blocks");
#define TR8(o, i, off) "ds_read_b64_tr_b8 %" #o ", %" #i " offset:" #off "\n\t"
  asm volatile(TR8(0, 8, 0) TR8(1, 9, 0) TR8(2, 8, 4096) TR8(3, 9, 4096) TR8(4, 8, 8192) TR8(5, 9, 8192) TR8(6, 8, 12288)
                   TR8(7, 9, 12288) "s_waitcnt lgkmcnt(0)"
               : "=&v"(f[0][0]), "=&v"(f[0][1]), "=&v"(f[1][0]), "=&v"(f[1][1]), "=&v"(f[2][0]), "=&v"(f[2][1]),
                 "=&v"(f[3][0]), "=&v"(f[3][1])
               : "v"(a[0]), "v"(a[1]));
#undef TR8
}
}  // namespace s8

// column tile nt over split z, as splitnn_dma_tile
template <int BR, int NS_>
__device__ __forceinline__ void grad8_tile(char* smem, const Act8Args& p, const int nt, const int z) {
  using namespace s8;
  using C = Cfg<BR, NS_>;
  constexpr int NS = C::NS, LEAD = NS - 1, FM = C::FM, FN = C::FN;
  asm volatile("" ::: "a0");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, hh = lane >> 5;
  const int64_t n0 = (int64_t)nt * BN;
  const int64_t kbeg = (int64_t)z * p.gksplit;
  const int64_t kend = kbeg + p.gksplit < p.M ? kbeg + p.gksplit : p.M;
  const int klen = kend > kbeg ? (int)(kend - kbeg) : 0;
  const int nk = (klen + BK - 1) / BK;

  const int dce = (lane & 7) ^ (lane >> 4), dco = (lane & 7) ^ ((lane >> 4) | 4);
  const char* ga = reinterpret_cast<const char*>(p.Qt) + kbeg * 2;
  const char* gb = reinterpret_cast<const char*>(p.codes) + kbeg * p.d + n0;
  const int64_t ncols = p.d - n0;
  auto dma = [&](const char* base, char* dst, bool ok, uint32_t off) {
    uint32_t vo = ok ? off : w4::OOB;
    asm volatile("" : "+v"(vo));
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, w4::BIG, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, (int)vo, 0, 0, 0);
  };
  auto issue = [&](int u) {
    char* st = smem + (u % NS) * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::IA; ++i) {
      const int row = 8 * (i + C::IA * wave) + (lane >> 3), kk = u * BK + 8 * (i & 1 ? dco : dce);
      dma(ga, st + 8 * (i + C::IA * wave) * 128, kk < klen && row < p.qr, (uint32_t)((row * p.rows + kk) * 2));
    }
    // instruction i of wave w: token rows 16 w + 4 i + lane / 16, the lane landing at chunk lane % 16
#pragma unroll
    for (int i = 0; i < C::IB; ++i) {
      const int k = 16 * wave + 4 * i + (lane >> 4), c = (lane & 15) ^ (2 * (k & 7));
      const char* base = gb + (int64_t)u * BK * p.d;
      dma(base, st + C::A_BYTES + (16 * wave + 4 * i) * 256, u * BK + k < klen && 16 * c < ncols, (uint32_t)(k * p.d + 16 * c));
    }
  };

  const int swz = (l32 >> 1) & 7;
  const uint32_t ra = (uint32_t)l32 * 128;
  // Lane l's fragment: column 32 j + l % 32, tokens 8 (l / 32) .. +7 of the step:
  // group gq = l / 16 reads columns 16 (2 j + (gq & 1)) .. and rows 8 (gq / 2) ..
  uint32_t rbo[FN];
  {
    const int gq = lane >> 4, i16 = lane & 15;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int chunk = 4 * wave + 2 * j + (gq & 1);
      rbo[j] = (uint32_t)C::A_BYTES + (uint32_t)(8 * (gq >> 1) + (i16 >> 1)) * 256 + (uint32_t)((chunk ^ (2 * (i16 >> 1))) << 4) +
               (uint32_t)((i16 & 1) << 3);
    }
  }
  f32x16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  if (nk > 0) {
#pragma unroll
    for (int u = 0; u < LEAD; ++u) issue(u);
    for (int t = 0; t < nk; ++t) {
      __builtin_amdgcn_s_waitcnt(pdma::vmcnt_imm(C::PER * (LEAD - 1)));
      lds_barrier();
      issue(t + LEAD);
      const char* st = smem + (t % NS) * C::STAGE;
      bf16x8 fa[4][FM];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[s][i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(st + ra + (((2 * s + hh) ^ swz) << 4) + i * 32 * 128));
      u32x2 fc[4][FN];
      const uint32_t ad[FN] = {lds_addr(st + rbo[0]), lds_addr(st + rbo[1])};
      tr_codes<FN>(fc, ad);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const bf16x8 fb = expand8(fc[s][j]);
#pragma unroll
          for (int i = 0; i < FM; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[s][i], fb, acc[i][j], 0, 0, 0);
        }
    }
    __builtin_amdgcn_s_waitcnt(pdma::vmcnt_imm(0));
  }
  float* out = p.gpart + (int64_t)z * p.qr * p.d;
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int row = 32 * i + 8 * (v >> 2) + 4 * hh + (v & 3);
      if (row >= p.qr) continue;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int64_t col = n0 + 64 * wave + 32 * j + l32;
        if (col < p.d) out[row * p.d + col] = acc[i][j][v];
      }
    }
}

struct Act8Pair {
  Act8Args a;
  GemmArgs g;
};

template <int BN>
__global__ void __launch_bounds__(pdma::NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
act8_panel_kernel(const Act8Pair q) {
  constexpr int L0 = p8::Cfg<BN>::LDS, L1 = pdma::Cfg<PANEL_BM, BN>::LDS;
  __shared__ __attribute__((aligned(1024))) char smem[L0 > L1 ? L0 : L1];
  const int y = (int)blockIdx.y;
  if (y < q.a.splits)
    panel8_tile<BN>(smem, q.a, (int)blockIdx.x, y);
  else
    panel_dma_tile<PANEL_BM, BN>(smem, q.g, (int)blockIdx.x, y - q.a.splits);
}

template <int BR, int NS8, int NS>
__global__ void __launch_bounds__(sdma::NT) __attribute__((amdgpu_waves_per_eu(1, 2)))
act8_grad_kernel(const Act8Pair q) {
  constexpr int L0 = s8::Cfg<BR, NS8>::LDS, L1 = sdma::Cfg<BR, NS>::LDS;
  __shared__ __attribute__((aligned(1024))) char smem[L0 > L1 ? L0 : L1];
  const int y = (int)blockIdx.y;
  const bool w = y >= q.a.gsplits;
  if ((int64_t)blockIdx.x * sdma::BN >= (w ? q.g.n_store : q.a.d)) return;
  if (!w)
    grad8_tile<BR, NS8>(smem, q.a, (int)blockIdx.x, y);
  else
    splitnn_dma_tile<BR, NS>(smem, q.g, (int)blockIdx.x, y - q.a.gsplits);
}

bool args_ok(const Act8Args& a) {
  return act8_fits(a.d, a.r8) && a.M > 0 && a.rows >= a.M && a.rows <= INT32_MAX && a.r <= a.r8 && a.splits >= 1 && a.gsplits >= 1 &&
         a.ksplit % 128 == 0 && a.gksplit % 64 == 0;
}

}  // namespace

// (lane offsets within a tile below the resource range)
bool act8_fits(int64_t d, int64_t r8) { return d % 16 == 0 && r8 <= 128 && d * 2 * 128 < (int64_t)w4::BIG; }

hipError_t launch_act8_panel_pair(const Act8Args& a, const GemmArgs& b, int sb, hipStream_t st) {
  if (!args_ok(a) || sb < 1 || b.n_store != a.r8 || b.m_store != a.rows || b.K2 || b.n_src || !panel_dma_fits(b.n_store, b.lda1, b.ldb1))
    return hipErrorInvalidValue;
  const dim3 grid((unsigned)((a.rows + PANEL_BM - 1) / PANEL_BM), (unsigned)(a.splits + sb));
  const Act8Pair q{a, b};
  if (a.r8 <= 64)
    hipLaunchKernelGGL((act8_panel_kernel<64>), grid, dim3(pdma::NT), 0, st, q);
  else
    hipLaunchKernelGGL((act8_panel_kernel<128>), grid, dim3(pdma::NT), 0, st, q);
  return hipGetLastError();
}

hipError_t launch_act8_grad_pair(const Act8Args& a, const GemmArgs& b, int sb, hipStream_t st) {
  // (the tokens' stride of Qt, and b as launch_gemm_pair checks it)
  if (!args_ok(a) || sb < 1 || a.rows * 2 * 128 >= (int64_t)w4::BIG || b.m_store != a.qr || (a.qr != a.r8 && a.qr != 2 * a.r8) || a.qr > 128 || b.m_load > b.m_store || b.n_load != b.n_store ||
      b.K2 || (b.k_split + sdma::BK) * b.ldb1 * 2 + b.n_store * 2 >= (int64_t)w4::BIG || b.lda1 * 2 * 128 >= (int64_t)w4::BIG)
    return hipErrorInvalidValue;
  const int64_t t0 = (a.d + s8::BN - 1) / s8::BN, t1 = (b.n_store + sdma::BN - 1) / sdma::BN;
  const dim3 grid((unsigned)std::max(t0, t1), (unsigned)(a.gsplits + sb));
  const Act8Pair q{a, b};
  // two blocks a CU where there are blocks for them, as the pair of bf16 ones
  if (a.qr <= 64 && t0 * a.gsplits + t1 * sb > 256)
    hipLaunchKernelGGL((act8_grad_kernel<64, 3, 2>), grid, dim3(sdma::NT), 0, st, q);
  else if (a.qr <= 64)
    hipLaunchKernelGGL((act8_grad_kernel<64, 6, 4>), grid, dim3(sdma::NT), 0, st, q);
  else
    hipLaunchKernelGGL((act8_grad_kernel<128, 5, 3>), grid, dim3(sdma::NT), 0, st, q);
  return hipGetLastError();
}

}  // namespace lora
