// gemm_w4_half.h - the NT GEMM on 128 x 256 tiles, 4 waves of 64 x 128, with
// the bias / activation / residual epilogue (epi.h):
//
//     C = act(A1 B1^T + A2 B2^T + bias) + residual
//
// for outputs of up to one such tile a CU.
//
// Tiles go to LDS by DMA as in gemm_w4_nt.h (same rows, swizzle and fragment
// reads), into a ring of 3 stages of 48 KiB: A's 128 rows of 128 bytes, then
// B's 256.  Stage t runs four contraction steps of 8 MFMAs:
//   step 0: reads of step 1's fragments; DMA of A(t+2)
//   step 1: reads of step 2's fragments; DMA of half of B(t+2)
//   step 2: reads of step 3's fragments; DMA of the other half
//   wait for this wave's DMAs of stage t+1 (vmcnt: only t+2's 12 may still
//   fly), barrier
//   step 3: reads of stage t+1's step-0 fragments
// Stage t+2's slot is stage t-1's, whose last reads came before the barrier
// of stage t-1.
//
// Ragged edges: a tile's rows past M (or N) are cut off by the buffer
// resource's length, so they read zeros, and are not stored; a last stage of
// fewer than 64 columns takes offsets past the resource for the others.
//
// Why this tile.  2048 x 4096 outputs are 256 of them and 128 of 256 x 256,
// which leave half of the CUs idle or have to be cut along the contraction.
// A 64 x 128 wave tile reads LDS 1.5 times as much a product as a 128 x 128
// one, which costs nothing at the power the chip has: 0.81 us a stage with 256
// blocks, 1325 TFLOP/s, 0.6 to 0.7 us with 128 or fewer.  A tile's launch,
// first stages and epilogue are 16 us.  Measured (MI355X, SiLU and residual, r =
// 16): 2048 x 4096 over 1024 27 us, over 2048 41, over 4096 68 (76 with two
// blocks for each 256 x 256 tile), 1024 x 4096 over 4096 50.  What bounds it:
// the power, then the fixed part.  Requesting A a quarter of a stage earlier
// gained nothing and its longer tail cost 3 us; blocks in the order of their
// numbers, without the XCDs' bands below, took 56 us for 1024 x 4096 over 4096.
#pragma once

#include "gemm_w4_nt.h"

namespace lora {

namespace w4h {
constexpr int BM = 128, FM = 2, TM = 64;
constexpr int A_BYTES = BM * 128, STAGE = A_BYTES + w4::BN * 128, NS = 3;
constexpr int LDS = NS * STAGE;
static_assert(LDS <= 160 * 1024, "the ring fits the LDS");
}  // namespace w4h

// Block b's tile.  Each of the 8 XCDs (which take blocks in turn) gets
// consecutive positions of an order of bands of 8 tile rows, each band column
// by column: 32 of them share 1024 rows of A and 1024 of B.
__device__ __forceinline__ void w4h_tile(int b, int blocks, int tm, int tn, int& mt, int& nt) {
  const int x = b & 7, q = blocks >> 3, rem = blocks & 7;
  const int e = x * q + min(x, rem) + (b >> 3);
  const int band = e / (8 * tn), in = e - band * 8 * tn, rows = min(8, tm - 8 * band);
  nt = in / rows;
  mt = 8 * band + in - nt * rows;
}

template <int EPI, bool MULTI = false>
__global__ void __launch_bounds__(w4::NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
gemm_w4_half_kernel(const GemmArgs p) {
  using w4::BN;
  using w4::FN;
  using w4::TN;
  using w4h::BM;
  using w4h::FM;
  using w4h::NS;
  using w4h::STAGE;
  using w4h::TM;
  using w4nt::vmcnt_imm;
  constexpr int BKS = w4nt::BK;
  static_assert(EPI == EPI_ACT, "the epilogue of epi.h");
  __shared__ __attribute__((aligned(1024))) char smem[w4h::LDS];
  // keep the MFMA accumulators in the accumulation registers
  asm volatile("" ::: "a0");

  const int n1 = (int)(p.K1 / BKS), kt = (int)(p.K1 % BKS);  // whole stages of the main segment, columns of a last one
  const int n1t = n1 + (kt ? 1 : 0);

  int mt, nt;
  w4h_tile((int)blockIdx.x, (int)gridDim.x, p.tiles_m, (int)((p.n_store + BN - 1) / BN), mt, nt);
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  const int64_t m0 = (int64_t)mt * BM, n0 = (int64_t)nt * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // A instruction i (< 4) of wave w moves rows 32 w + 8 i + lane / 8, B instruction
  // i (< 8) rows 64 w + 8 i + lane / 8
  const int rowa = 32 * wave + (lane >> 3), rowb = 64 * wave + (lane >> 3);
  // MULTI: the tile's adapters, and those of the rows that this lane moves
  int ads = 0;
  uint32_t adl[1], rad[2];
  if constexpr (MULTI) {
    ads = scalar_at(p.ad_cnt, mt);
    ad_load_list(p, mt, ads, lane, adl);
    ad_load_rows(p, m0 + rowa, rad);
  }
  const int rank2 = MULTI ? ads * p.ad_r : (int)p.K2;  // columns of the second segment
  const int n = n1t + (rank2 + BKS - 1) / BKS;

  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using T_ = std::true_type;
  using F_ = std::false_type;

  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, hh = lane >> 5;
  const int dce = (lane & 7) ^ (lane >> 4), dco = (lane & 7) ^ ((lane >> 4) | 4);
  const uint32_t ra1 = (uint32_t)(rowa * p.lda1 * 2), ra2 = (uint32_t)(rowa * p.lda2 * 2);
  const uint32_t rb1 = (uint32_t)(rowb * p.ldb1 * 2), rb2 = (uint32_t)(rowb * p.ldb2 * 2);
  const uint32_t va1[2] = {ra1 + (uint32_t)(dce * 16), ra1 + (uint32_t)(8 * p.lda1 * 2 + dco * 16)};
  const uint32_t vb1[2] = {rb1 + (uint32_t)(dce * 16), rb1 + (uint32_t)(8 * p.ldb1 * 2 + dco * 16)};
  const uint32_t isa1 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.lda1 * 2));
  const uint32_t isa2 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.lda2 * 2));
  const uint32_t isb1 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.ldb1 * 2));
  const uint32_t isb2 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.ldb2 * 2));
  const uint32_t oda2 = (uint32_t)(8 * p.lda2 * 2), odb2 = (uint32_t)(8 * p.ldb2 * 2);
  const int k2 = __builtin_amdgcn_readfirstlane((int)p.K2);

  const uint32_t ra = (uint32_t)(wm * TM + l32) * 128;
  const uint32_t rb = (uint32_t)w4h::A_BYTES + (uint32_t)(wn * TN + l32) * 128;
  const int swz = (l32 >> 1) & 7;
  bf16x8 fa[2][FM], fb[2][FN];
  auto rd1 = [&](int st, int s, auto fsel, int k) {
    constexpr int f = decltype(fsel)::value;
    const uint32_t c = (uint32_t)(((2 * s + hh) ^ swz) << 4);
    if (k < FM)
      fa[f][k] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(smem + st * STAGE + ra + c + k * 32 * 128));
    else
      fb[f][k - FM] =
          __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(smem + st * STAGE + rb + c + (k - FM) * 32 * 128));
  };
  f32x16 acc[FM][FN];
  auto mf = [&](auto fsel, int q) {
    constexpr int f = decltype(fsel)::value;
    acc[q >> 2][q & 3] =
        __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[f][q >> 2], fb[f][q & 3], acc[q >> 2][q & 3], 0, 0, 0);
  };

  const char* ga1 = reinterpret_cast<const char*>(p.a1) + m0 * p.lda1 * 2;
  const char* ga2 = reinterpret_cast<const char*>(p.a2) + m0 * p.lda2 * 2;
  const char* gb1 = reinterpret_cast<const char*>(p.b1) + n0 * p.ldb1 * 2;
  const char* gb2 = reinterpret_cast<const char*>(p.b2) + n0 * p.ldb2 * 2;
  // bytes from ga1 (gb1, ..) to the end of the tile's last existing row
  const int ma = (int)min(p.m_load - m0, (int64_t)BM), nb = (int)min(p.n_load - n0, (int64_t)BN);
  const int la1 = (int)(ma * p.lda1 * 2), la2 = (int)(ma * p.lda2 * 2);
  const int lb1 = (int)(nb * p.ldb1 * 2), lb2 = (int)(nb * p.ldb2 * 2);

  // MULTI: the lane's rows of a strip and of the second operand, in bytes; the latter's end
  const uint32_t isr = (uint32_t)(p.ad_r * 2), ar2 = rowa * isr, br2 = rowb * isr;
  const int adlen = MULTI ? (int)(uint32_t)(p.ad_n * p.ad_step * 2 - n0 * p.ldb2 * 2) : 0;
  auto seg_of = [&](int u) {
    if constexpr (MULTI)
      return ad_seg(p, adl, ads, u - n1t, dce, dco);
    else
      return AdSeg{};
  };

  // One DMA: stage u, operand op (0 A, 1 B), instruction i, ring stage s.
  auto dma = [&](int u, int s, int op, int i, auto seg2_c, const AdSeg& sg) {
    constexpr bool SEG2 = decltype(seg2_c)::value;
    const int odd = i & 1, pair = i >> 1;
    const char* base;
    int len;
    uint32_t vo, is;
    if constexpr (!SEG2) {
      base = (op == 0 ? ga1 : gb1) + (int64_t)u * (BKS * 2);
      len = (op == 0 ? la1 : lb1) - u * (BKS * 2);
      vo = op == 0 ? va1[odd] : vb1[odd];
      is = op == 0 ? isa1 : isb1;
    } else {
      const int tt = u - n1t;
      const int dc = odd ? dco : dce;
      if (tt < 0) {  // the main segment's last columns
        base = (op == 0 ? ga1 : gb1) + (int64_t)u * (BKS * 2);
        len = (op == 0 ? la1 : lb1) - u * (BKS * 2);
        vo = 8 * dc < kt ? (op == 0 ? va1[odd] : vb1[odd]) : w4::OOB;
        is = op == 0 ? isa1 : isb1;
      } else if constexpr (MULTI) {
        if (op == 0) {
          base = ga2;
          len = la2;
          vo = (rad[(i >> 1) & 1] >> (16 * (i & 1)) & 0xFFFFu) == sg.a[odd] ? ar2 + (uint32_t)(8 * i) * isr + sg.q[odd] : AD_OOB;
        } else {  // (rows past the last read the next adapter's, into columns that are not stored)
          base = gb2;
          len = adlen;
          vo = sg.b[odd] + br2 + (uint32_t)(8 * i) * isr;
        }
        is = 0;
      } else {
        const int kk = tt * BKS + 8 * dc;  // the lane's first rank column
        const uint32_t kc = (uint32_t)(tt * BKS * 2 + dc * 16);
        base = op == 0 ? ga2 : gb2;
        len = op == 0 ? la2 : lb2;
        vo = kk < k2 ? (op == 0 ? ra2 + (odd ? oda2 : 0u) : rb2 + (odd ? odb2 : 0u)) + kc : w4::OOB;
        is = op == 0 ? isa2 : isb2;
      }
    }
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, len, 0x00020000);
    char* dst = smem + s * STAGE + (op == 0 ? (4 * wave + i) * 1024 : w4h::A_BYTES + (8 * wave + i) * 1024);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)dst, 16, (int)(vo + (uint32_t)pair * is), 0, 0, 0);
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // prologue: stages 0 and 1 in flight; wait for stage 0
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (u < n1) {
#pragma unroll
      for (int i = 0; i < 12; ++i) dma(u, u, i < 4 ? 0 : 1, i < 4 ? i : i - 4, F_{}, AdSeg{});
    } else if (u < n) {
      const AdSeg sg = seg_of(u);
#pragma unroll
      for (int i = 0; i < 12; ++i) dma(u, u, i < 4 ? 0 : 1, i < 4 ? i : i - 4, T_{}, sg);
    }
  }
  if (n >= 2)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(12));
  else
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  lds_barrier();
#pragma unroll
  for (int k = 0; k < 6; ++k) rd1(0, 0, I0{}, k);

  // One stage.  ISSUE: 0 none, 1 a whole stage t+2 of the main segment, 2 its
  // ragged last one or one of the rank segment.  NEXT: stage t+1 exists.
  auto stage = [&](int t, auto issue_c, auto next_c) {
    constexpr int ISSUE = decltype(issue_c)::value;
    constexpr bool NEXT = decltype(next_c)::value;
    using S2 = std::integral_constant<bool, ISSUE == 2>;
    const AdSeg sg = ISSUE == 2 ? seg_of(t + 2) : AdSeg{};
    const int s = t % NS, s1 = (t + 1) % NS, s2 = (t + 2) % NS;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      mf(I0{}, q);
      if (q < 6) rd1(s, 1, I1{}, q);
      if (ISSUE && (q & 1)) dma(t + 2, s2, 0, q >> 1, S2{}, sg);
      fence();
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      mf(I1{}, q);
      if (q < 6) rd1(s, 2, I0{}, q);
      if (ISSUE && (q & 1)) dma(t + 2, s2, 1, q >> 1, S2{}, sg);
      fence();
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      mf(I0{}, q);
      if (q < 6) rd1(s, 3, I1{}, q);
      if (ISSUE && (q & 1)) dma(t + 2, s2, 1, 4 + (q >> 1), S2{}, sg);
      fence();
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(ISSUE ? 12 : 0));
    lds_barrier();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      mf(I1{}, q);
      if (NEXT && q < 6) rd1(s1, 0, I0{}, q);
      fence();
    }
  };
  using N0 = std::integral_constant<int, 0>;
  using N1 = std::integral_constant<int, 1>;
  using N2 = std::integral_constant<int, 2>;
  int t = 0;
  for (; t + 2 < n1; ++t) stage(t, N1{}, T_{});
  for (; t + 2 < n; ++t) stage(t, N2{}, T_{});
  if (t + 1 < n) stage(t++, N0{}, T_{});
  stage(t, N0{}, F_{});

  w4_epilogue<EPI, true, FM>(p, acc, smem, m0, n0, p.c, p.ldc);
}

}  // namespace lora
