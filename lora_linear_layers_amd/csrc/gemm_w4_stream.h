// gemm_w4_stream.h - the whole-tile NT GEMM's main loop (gemm_w4_nt.h: 256 x
// 256 tiles, 4 waves of 128 x 128, tiles DMA'd into a 5-slot LDS ring) for
// outputs whose tiles are neither whole nor a multiple of the CUs, with the
// bias / activation / residual epilogue (epi.h):
//
//     C = act(A1 B1^T + A2 B2^T + bias) + residual
//
// Ragged edges: a tile's rows past M (or N) are cut off by the buffer
// resource's length, so they read zeros, and are not stored; a last stage of
// fewer than 64 columns takes offsets past the resource for the others.
//
// Work split: the first st_full tiles are a block each; each of the st_half
// tiles after them is two blocks, the first and the second part of its
// contraction, so that 64 to 128 tiles fill 256 CUs (2048 x 4096 outputs are
// 128; up to 224 stages gemm_w4_half.h takes those).  A part's block leaves
// its accumulators in its slot, in the registers' order, and counts itself in;
// the one that comes second adds the other's slot as it stages the rows of its
// epilogue (a sum of two does not depend on their order) and stores.  Nobody
// waits for anybody.  The first part is `st_early` stages short of half and the
// second as much longer, so that the first's slot is usually there when the
// second ends, which then writes none.
//
// Slots, counters: fp32 [2 st_half][256 * 256] and int [st_half], zero before
// the launch.  They cross XCDs, so they are written and read at the device's
// coherence point (sc1 stores and loads, as in few.h), each block's stores
// complete before it counts itself in.
// What it measures (MI355X, r = 16 to 64, bias / SiLU / residual): a tile alone
// on its CU costs 18.5 us (launch, first stages, epilogue) and 1.1 to 1.5 us a
// 64-deep stage, with 128 to 256 CUs at work; two blocks a tile 37 us and 0.66 us
// a stage.  2049 x 4104 over 4096 (153 tiles): 86 us (91 in a sustained loop, 101
// in its first calls), 34 % of the chip's MFMA cycles, 60 % of its CUs; 2048 x 4096 over 4096 (128 tiles in two): 76 us, 39 %;
// over 14336: 197 us.  What bounds it: the CUs without a tile, then the fixed
// part; contiguous ranges that span tiles (three slots of 256 KB to read back
// for some) and no stagger between the parts measured slower (137 and 85 us
// against 86 and 76); tiles in bands by XCD gained nothing (2049 x 4104 over 4096:
// 109 us a pass against 108).
#pragma once

#include "gemm_w4_nt.h"

namespace lora {

template <int EPI>
__global__ void __launch_bounds__(w4::NT) __attribute__((amdgpu_waves_per_eu(1, 1)))
gemm_w4_stream_kernel(const GemmArgs p) {
  using namespace w4;
  using w4nt::NSLOT;
  using w4nt::SLOT;
  using w4nt::vmcnt_imm;
  constexpr int BKS = w4nt::BK;
  static_assert(EPI == EPI_ACT, "the epilogue of epi.h");
  __shared__ __attribute__((aligned(1024))) char smem[w4nt::LDS];
  // keep the MFMA accumulators in the accumulation registers
  asm volatile("" ::: "a0");

  const int nk1 = (int)(p.K1 / BKS), kt = (int)(p.K1 % BKS);  // whole stages of the main segment, columns of a last one
  const int nk1t = nk1 + (kt ? 1 : 0);
  const int nk = nk1t + (int)((p.K2 + BKS - 1) / BKS);

  // the block's tile and its stages [s0, s0 + n) of it
  const int bid = blockIdx.x, hb = bid - p.st_full;
  const bool part = hb >= 0;
  const int tile = part ? p.st_full + (hb >> 1) : bid;
  const int mid = nk / 2 - p.st_early;
  const int s0 = part && (hb & 1) ? mid : 0;
  const int n = part ? (hb & 1 ? nk - mid : mid) : nk;

  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using T_ = std::true_type;
  using F_ = std::false_type;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, hh = lane >> 5;
  const int dr = lane >> 3;
  const int dce = (lane & 7) ^ (lane >> 4), dco = (lane & 7) ^ ((lane >> 4) | 4);
  const int row0 = 64 * wave + dr;
  const uint32_t ra1 = (uint32_t)(row0 * p.lda1 * 2), ra2 = (uint32_t)(row0 * p.lda2 * 2);
  const uint32_t rb1 = (uint32_t)(row0 * p.ldb1 * 2), rb2 = (uint32_t)(row0 * p.ldb2 * 2);
  const uint32_t va1[2] = {ra1 + (uint32_t)(dce * 16), ra1 + (uint32_t)(8 * p.lda1 * 2 + dco * 16)};
  const uint32_t vb1[2] = {rb1 + (uint32_t)(dce * 16), rb1 + (uint32_t)(8 * p.ldb1 * 2 + dco * 16)};
  const uint32_t isa1 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.lda1 * 2));
  const uint32_t isa2 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.lda2 * 2));
  const uint32_t isb1 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.ldb1 * 2));
  const uint32_t isb2 = __builtin_amdgcn_readfirstlane((uint32_t)(16 * p.ldb2 * 2));
  const uint32_t oda2 = (uint32_t)(8 * p.lda2 * 2), odb2 = (uint32_t)(8 * p.ldb2 * 2);
  const int k2 = __builtin_amdgcn_readfirstlane((int)p.K2);

  const uint32_t ra = (uint32_t)(wm * TM + l32) * 128;
  const uint32_t rb = (uint32_t)(wn * TN + l32) * 128;
  const int swz = (l32 >> 1) & 7;
  bf16x8 fa[2][FM], fb[2][FN];
  auto rd1 = [&](int sa, int sbl, int s, auto fsel, int k) {
    constexpr int f = decltype(fsel)::value;
    const uint32_t c = (uint32_t)(((2 * s + hh) ^ swz) << 4);
    if (k < FM)
      fa[f][k] = __builtin_bit_cast(bf16x8,
                                    *reinterpret_cast<const u32x4*>(smem + sa * SLOT + ra + c + k * 32 * 128));
    else
      fb[f][k - FM] = __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(smem + sbl * SLOT + rb + c + (k - FM) * 32 * 128));
  };
  f32x16 acc[FM][FN];
  auto mf = [&](auto fsel, int q) {
    constexpr int f = decltype(fsel)::value;
    acc[q >> 2][q & 3] =
        __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[f][q >> 2], fb[f][q & 3], acc[q >> 2][q & 3], 0, 0, 0);
  };

  const int64_t m0 = (int64_t)(tile % p.tiles_m) * BM;
  const int64_t n0 = (int64_t)(tile / p.tiles_m) * BN;
  const int n1 = max(0, min(nk1 - s0, n));  // stages of the main segment
  const char* ga1 = reinterpret_cast<const char*>(p.a1) + m0 * p.lda1 * 2 + (int64_t)s0 * (BKS * 2);
  const char* ga2 = reinterpret_cast<const char*>(p.a2) + m0 * p.lda2 * 2;
  const char* gb1 = reinterpret_cast<const char*>(p.b1) + n0 * p.ldb1 * 2 + (int64_t)s0 * (BKS * 2);
  const char* gb2 = reinterpret_cast<const char*>(p.b2) + n0 * p.ldb2 * 2;
  // bytes from ga1 (gb1, ..) to the end of the tile's last existing row
  const int ma = (int)min(p.m_load - m0, (int64_t)BM), nb_ = (int)min(p.n_load - n0, (int64_t)BN);
  const int la1 = (int)(ma * p.lda1 * 2) - s0 * (BKS * 2), la2 = (int)(ma * p.lda2 * 2);
  const int lb1 = (int)(nb_ * p.ldb1 * 2) - s0 * (BKS * 2), lb2 = (int)(nb_ * p.ldb2 * 2);

  // One DMA: the block's stage u, operand op (0 A, 1 B), instruction i (< 8),
  // slot s.
  auto dma = [&](int u, int s, int op, int i, auto seg2_c) {
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
      const int tt = s0 + u - nk1t;
      const int dc = odd ? dco : dce;
      if (tt < 0) {  // the main segment's last columns
        base = (op == 0 ? ga1 : gb1) + (int64_t)u * (BKS * 2);
        len = (op == 0 ? la1 : lb1) - u * (BKS * 2);
        vo = 8 * dc < kt ? (op == 0 ? va1[odd] : vb1[odd]) : w4::OOB;
        is = op == 0 ? isa1 : isb1;
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
    char* dst = smem + s * SLOT + (8 * wave + i) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)dst, 16, (int)(vo + (uint32_t)pair * is), 0, 0, 0);
  };

#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

  // prologue: stages 0 and 1 in flight (slots 0 .. 3); wait for stage 0
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (u < n1) {
#pragma unroll
      for (int i = 0; i < 16; ++i) dma(u, 2 * u + (i >> 3), i >> 3, i & 7, F_{});
    } else if (u < n) {
#pragma unroll
      for (int i = 0; i < 16; ++i) dma(u, 2 * u + (i >> 3), i >> 3, i & 7, T_{});
    }
  }
  if (n >= 2)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(16));
  else
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  lds_barrier();
#pragma unroll
  for (int k = 0; k < 8; ++k) rd1(0, 1, 0, I0{}, k);

  // One stage, as in gemm_w4_nt_kernel.  ISSUE: 0 none, 1 a whole stage t+2 of
  // the main segment, 2 its ragged last one or one of the rank segment.  NEXT: stage t+1 exists.
  auto stage = [&](int t, auto issue_c, auto next_c) {
    constexpr int ISSUE = decltype(issue_c)::value;
    constexpr bool NEXT = decltype(next_c)::value;
    using S2 = std::integral_constant<bool, ISSUE == 2>;
    const int sa = (2 * t) % NSLOT, sbl = (2 * t + 1) % NSLOT;
    const int na = (2 * t + 2) % NSLOT, nb = (2 * t + 3) % NSLOT;
    const int fa2 = (2 * t + 4) % NSLOT;  // A(t+2): the slot of B(t-1)
    const int fb2 = sa;                   // B(t+2): the slot of A(t)
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      mf(I0{}, q);
      if (q < 8)
        rd1(sa, sbl, 1, I1{}, q);
      else if (ISSUE && (q & 1) == 0)
        dma(t + 2, fa2, 0, (q - 8) >> 1, S2{});
      fence();
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      mf(I1{}, q);
      if (q < 8)
        rd1(sa, sbl, 2, I0{}, q);
      else if (ISSUE && (q & 1) == 0)
        dma(t + 2, fa2, 0, 4 + ((q - 8) >> 1), S2{});
      fence();
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      mf(I0{}, q);
      if (q < 8) rd1(sa, sbl, 3, I1{}, q);
      fence();
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(ISSUE ? 8 : 0));
    lds_barrier();
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      mf(I1{}, q);
      if (q < 8) {
        if (NEXT) rd1(na, nb, 0, I0{}, q);
      } else if (ISSUE) {
        dma(t + 2, fb2, 1, q - 8, S2{});
      }
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

  const float* other = nullptr;
  if (part) {
    int* cnt = p.st_cnt + (hb >> 1);
    int* second = reinterpret_cast<int*>(smem);  // (between the last reads of the ring and its next use)
    if (tid == 0) *second = __hip_atomic_load(cnt, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (!*second) {
      const __amdgpu_buffer_rsrc_t mine = __builtin_amdgcn_make_buffer_rsrc(
          p.st_part + (int64_t)hb * (BM * BN), (short)0, BM * BN * 4, 0x00020000);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), mine,
                                                   ((i * FN + j) * 4 + q) * (NT * 16) + tid * 16, 0, 16);
          }
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // this wave's part is in memory
      __syncthreads();                           // and the other waves'
      if (tid == 0) *second = __hip_atomic_fetch_add(cnt, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      if (!*second) return;
    }
    asm volatile("" ::: "memory");
    other = p.st_part + (int64_t)(hb ^ 1) * (BM * BN);
  }
  w4_epilogue<EPI, true>(p, acc, smem, m0, n0, p.c, p.ldc, other);
}

}  // namespace lora
