// kepttile.hpp -- tiles of dw = dy^T x~, x~ the kept activations (e4m3 codes, a
// power of two for each 32 tokens of a column), on the bf16 matrix instructions.
//
// A workgroup of WM x WN waves takes a TM x TN tile (rows: columns of dy;
// columns: those of x~), each wave TM/WM x TN/WN of it in blocks of 32 x 32.  K
// are the tokens, 64 to a stage.  In LDS a stage is
//   dy:     panels of 64 columns, 64 rows of 128 bytes each, swizzled as the
//           GEMM's MN-contiguous operands (kernel/mainloop.hpp) and read with
//           transposing reads;
//   codes:  [4 groups of 16 tokens][TN columns][16 bytes], as in memory: a
//           fragment's 16 tokens of a column are one ds_read_b128, whose lanes
//           are contiguous;
//   powers: for each wave [2 groups of 32 tokens][its columns], a byte each.
// Lane l of a 32-token group holds tokens 16 (l / 32) .. + 15 of its column: the
// first eight for one k-step and the rest for the next.  dy's reads take the
// same tokens.  Which K the instructions take them for does not matter.
//
// Codes become bf16 in registers, a v_cvt_scalef32_pk_bf16_fp8 for each pair,
// which applies the power too: exact, and four of them to a fragment of eight.
// Half the bytes of a bf16 operand go through memory and LDS.
//
// Bound: the matrix instructions, busy in 73% of the cycles of 8192^3, at a clock
// that the board's power limit holds at 1.55 to 1.85 GHz.  Tiles that fill their
// rounds poorly and have few stages leave them idle: 2048 x 4096 x 11008 (928
// tiles of 32 stages, 3.6 rounds) 50%, 1001 x 2000 x 5000 (216 of 16) 29%.  With
// the codes taken for bf16 as they are the loop takes as long, so the conversions
// hide behind the products; without its loads it takes 15% less (256 x 256, 128
// stages: 126 us for 145).  The large tiles have eight waves, two a SIMD: one's
// products run while the other waits at the barrier or for its fragments.  With
// four, each with twice the blocks and all of a SIMD's registers, 1000^3 in one
// round of 192 x 256 took 23.3 us for 20.8 and 2048 x 4096 x 11008 186 for 180;
// the small tiles have their second workgroup for that (128 x 128 with eight
// waves: slower).
//
// The ring has SLOTS >= 3 stages.  An iteration begins behind the barrier that
// certifies stage d + 1 and frees stage d, whose last k-step is in registers:
// its 4 k-steps are that one and the first three of stage d + 1, each preparing
// the next one's fragments, and the loads of stage d + SLOTS are spread over all
// of them.  They have SLOTS - 2 iterations to land.
#pragma once

#include "../kernel/gfx950.hpp"
#include "../kernel/mainloop.hpp"
#include "midtile.hpp"
#include "operators.h"

namespace migemm {

constexpr int kKeptTokens = 64;  // a stage

template <int TM, int TN, int SLOTS, int WM, int WN>
struct KeptGeom {
  static constexpr int kWaves = WM * WN;
  static constexpr int kBM = TM / (32 * WM), kBN = TN / (32 * WN);  // a wave's 32 x 32 blocks
  static constexpr int kLoadsA = TM / (8 * kWaves), kLoadsB = TN / (16 * kWaves);
  static constexpr int kLoads = kLoadsA + kLoadsB + 1;  // of a wave and stage
  static constexpr uint32_t kCodes = TM * 128, kPowers = kCodes + TN * kKeptTokens, kSlot = kPowers + kWaves * 256;
  static constexpr uint32_t kRing = SLOTS * kSlot;
  // Epilogue staging, of each wave: bf16, all its rows; fp32, 32 at a time.
  static constexpr uint32_t kStaging16 = kWaves * 32 * kBM * (64 * kBN + 16), kStaging32 = kWaves * 32 * (128 * kBN + 16);
  static constexpr uint32_t kStaging = kStaging16 > kStaging32 ? kStaging16 : kStaging32;
  static constexpr uint32_t kLds = kRing > kStaging ? kRing : kStaging;
  static_assert(kLds <= kLdsLimit && (SLOTS - 2) * kLoads < 64, "the ring fits LDS, its loads vmcnt");
};

// dy's fragments: MidReader's, with the tokens of a 32-token group in the order
// above.  KS = 2 G + S: eight tokens S of group G.
template <int NB>
struct KeptReader {
  typedef StageGeom<2> G;
  uint32_t off[NB];
  __device__ __forceinline__ void init(int col0, int lane) {
    const int g = lane >> 4, t = lane & 15;
    const int k = 16 * (g >> 1) + (t >> 2);
    const int chunk = 2 * (g & 1) + ((t & 3) >> 1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int h = col0 / 32 + b;
      off[b] = (h >> 1) * G::kPanelBytes + k * kPanelRowBytes +
               (((4 * (h & 1) + chunk) ^ swz_mn<2>(k)) << 4) + 8 * (t & 1);
    }
  }
  template <int BLK, int KS>
  __device__ __forceinline__ bf16x8 read(uint32_t opnd) const {
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    constexpr uint32_t c = (32 * (KS >> 1) + 8 * (KS & 1)) * kPanelRowBytes;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MIGEMM_LDS i16x4*)lds_at(opnd + off[BLK] + c));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (MIGEMM_LDS i16x4*)lds_at(opnd + off[BLK] + c + 4 * kPanelRowBytes));
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
  }
};

// Eight codes of a column as bf16.
__device__ __forceinline__ bf16x8 kept_bf16(int w0, int w1, float power) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w0, power, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w0, power, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w1, power, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w1, power, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// dy's loads of a stage: MidLoader's layout, for any whole number of loads a
// wave.  Tokens past the last lie past dy's end, where loads give zeros, so no
// load needs a mask.
template <int NL>
struct KeptDyLoader {
  typedef StageGeom<2> G;
  uint64_t at;  // the next stage's
  int64_t left, step;
  uint32_t off[NL];
  __device__ __forceinline__ void init(const CheckpointArgs& a, int64_t m0, int stage, int wave, int lane) {
    step = (int64_t)kKeptTokens * a.dy_rs * 2;
    at = reinterpret_cast<uint64_t>(a.dy) + m0 * 2 + stage * step;
    // (Range checks work on dwords: up to the end of the last 16-byte block.)
    left = (((a.tokens - 1) * a.dy_rs + a.out_cols - m0) * 2 - stage * step + 15) & ~(int64_t)15;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int idx = wave * NL + j;  // 8 rows of a panel
      const int row = (idx % G::kLoadsPerPanel) * 8 + (lane >> 3);
      const int col = (idx / G::kLoadsPerPanel) * G::kPanelCols + ((lane & 7) ^ swz_mn<2>(row)) * G::kElemsPerChunk;
      off[j] = (uint32_t)((row * a.dy_rs + col) * 2);
    }
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t next() {
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(reinterpret_cast<const void*>(at), left < 0 ? 0 : (left > 0x7FFFFFF0 ? 0x7FFFFFF0u : (uint32_t)left));
    at += step, left -= step;
    return r;
  }
};

// The codes' and powers' loads of a stage.  Groups of tokens past the kept ones
// read as zero; columns past the last read other codes, or zeros, for columns
// of dw that are not stored.
template <int TN, int BN, int WN, int NL>
struct KeptLoader {
  uint64_t codes_at, powers_at;  // the next stage's
  int64_t codes_left, powers_left, ld;
  uint32_t code_off[NL], power_off;
  __device__ __forceinline__ void init(const CheckpointArgs& a, int64_t k0, int stage, int wave, int lane) {
    const int64_t groups = (a.tokens + 31) / 32;
    ld = a.ld;
    codes_at = reinterpret_cast<uint64_t>(a.codes) + ((int64_t)stage * 4 * ld + k0) * 16;
    codes_left = groups * 32 * ld - ((int64_t)stage * 4 * ld + k0) * 16;
    const int64_t col = k0 + wave % WN * 32 * BN;
    powers_at = reinterpret_cast<uint64_t>(a.scales) + (int64_t)stage * 2 * ld + col;
    powers_left = groups * ld - (int64_t)stage * 2 * ld - col;
#pragma unroll
    for (int j = 0; j < NL; ++j) {
      const int idx = wave * NL + j;  // 64 columns of a group
      code_off[j] = (uint32_t)(((idx / (TN / 64)) * ld + 64 * (idx % (TN / 64)) + lane) * 16);
    }
    constexpr int kLanes = 8 * BN;  // a group's columns, four a lane
    power_off = lane < 2 * kLanes ? (uint32_t)(lane / kLanes * ld + 4 * (lane % kLanes)) : kOobOffset;
  }
  struct Stage {
    __amdgpu_buffer_rsrc_t codes, powers;
  };
  __device__ __forceinline__ Stage next() {
    auto rsrc = [](uint64_t at, int64_t left) {
      return make_rsrc(reinterpret_cast<const void*>(at), left < 0 ? 0 : (left > 0x7FFFFFF0 ? 0x7FFFFFF0u : (uint32_t)left));
    };
    const Stage s = {rsrc(codes_at, codes_left), rsrc(powers_at, powers_left)};
    codes_at += 64 * ld, codes_left -= 64 * ld;
    powers_at += 2 * ld, powers_left -= 2 * ld;
    return s;
  }
};

// Stages [k0, k0 + KT) of the tile at (m0, n0).  On return every wave is done with the ring.
template <int TM, int TN, int SLOTS, int WM, int WN, class Acc>
__device__ __forceinline__ void kept_loop(Acc& acc, const CheckpointArgs& a, int64_t m0, int64_t n0, int wave,
                                          int lane, int k0, int KT) {
  typedef KeptGeom<TM, TN, SLOTS, WM, WN> T;
  constexpr int BM = T::kBM, BN = T::kBN, NLA = T::kLoadsA, NLB = T::kLoadsB, P = BM * BN;
  KeptDyLoader<NLA> la;
  KeptLoader<TN, BN, WN, NLB> lb;
  la.init(a, m0, k0, wave, lane);
  lb.init(a, n0, k0, wave, lane);
  KeptReader<BM> ra;
  ra.init(wave / WN * 32 * BM, lane);
  const uint32_t code_at = T::kCodes + ((lane >> 5) * TN + wave % WN * 32 * BN + (lane & 31)) * 16;
  const uint32_t power_at = T::kPowers + wave * 256 + (lane & 31);
#pragma unroll
  for (int i = 0; i < BM; ++i)
#pragma unroll
    for (int j = 0; j < BN; ++j) acc.v[i][j] = f32x16{};

  bf16x8 fa[2][BM], fb[2][BN];
  i32x4 raw[BN];
  uint32_t power[2][BN];
  // Piece x of preparing k-step KS of the stage in `slot`: what it reads (the
  // powers and codes where a stage or a group begins, then dy), then its codes'
  // conversion.
  auto prepare = [&](auto kc, auto xc, uint32_t slot) {
    constexpr int ks = decltype(kc)::value, x = decltype(xc)::value;
    constexpr int kPow = ks == 0 ? 2 * BN : 0, kRaw = kPow + (ks % 2 == 0 ? BN : 0), kDy = kRaw + BM;
    if constexpr (x < kPow) {
      power[x / BN][x % BN] = *(const MIGEMM_LDS unsigned char*)lds_at(slot + power_at + (x / BN) * 32 * BN + 32 * (x % BN));
    } else if constexpr (x < kRaw) {
      constexpr int j = x - kPow;
      raw[j] = *(const MIGEMM_LDS i32x4*)lds_at(slot + code_at + (ks >> 1) * 2 * TN * 16 + j * 512);
    } else if constexpr (x < kDy) {
      fa[ks & 1][x - kRaw] = ra.template read<x - kRaw, ks>(slot);
    } else {
      constexpr int j = x - kDy;
      fb[ks & 1][j] = kept_bf16(raw[j][2 * (ks & 1)], raw[j][2 * (ks & 1) + 1], __uint_as_float(power[ks >> 1][j] << 23));
    }
  };
  auto load = [&](const auto& sa, const auto& sb, auto jc, uint32_t slot) {
    constexpr int j = decltype(jc)::value;
    if constexpr (j < NLA) dma16(sa, lds_at(slot + (wave * NLA + j) * 1024), la.off[j]);
    else if constexpr (j < NLA + NLB) dma16(sb.codes, lds_at(slot + T::kCodes + (wave * NLB + j - NLA) * 1024), lb.code_off[j - NLA]);
    else dma4(sb.powers, lds_at(slot + T::kPowers + wave * 256), lb.power_off);
  };
  // The products of one k-step (buffer KS & 1) while the next one is prepared.
  auto step = [&](auto kc, uint32_t next_slot, auto&& behind) {
    constexpr int ks = decltype(kc)::value, next = (ks + 1) & 3;
    constexpr int n = (next == 0 ? 2 * BN : 0) + (next % 2 == 0 ? BN : 0) + BM + BN;
    static_for<0, P>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      sched_fence();
      static_for<m * n / P, (m + 1) * n / P>([&](auto xc) { prepare(std::integral_constant<int, next>{}, xc, next_slot); });
      acc.v[m / BN][m % BN] = mfma<2>(fb[ks & 1][m % BN], fa[ks & 1][m / BN], acc.v[m / BN][m % BN]);
      behind(mc);
    });
  };
  auto after = [](uint32_t slot) { return slot + T::kSlot == T::kRing ? 0 : slot + T::kSlot; };
  const auto nothing = [](auto) {};

  // Stages past KT load what lies there, or zeros, which nobody reads: the
  // count of loads in flight stays fixed.
  static_for<0, SLOTS>([&](auto sc) {
    const auto sa = la.next();
    const auto sb = lb.next();
    static_for<0, T::kLoads>([&](auto jc) { load(sa, sb, jc, decltype(sc)::value * T::kSlot); });
  });
  sched_fence();
  wait_vmcnt<(SLOTS - 1) * T::kLoads>();
  barrier();
  if (KT > 0) {
    static_for<0, 3 * BN + BM + BN>([&](auto xc) { prepare(std::integral_constant<int, 0>{}, xc, 0); });
    static_for<0, 3>([&](auto kc) { step(kc, 0, nothing); });
  }
  // (The last k-step comes after the loop: a way out inside it would let the
  // compiler move a fragment's conversion past its products.)
  uint32_t cur = 0;
  for (int d = 0; d + 1 < KT; ++d) {
    // Stage d + 1 has landed and this wave's reads of stage d have returned;
    // past the barrier that holds for every wave.
    sched_fence();
    wait_vmcnt<(SLOTS - 2) * T::kLoads>();
    wait_lgkmcnt<0>();
    barrier();
    const uint32_t nxt = after(cur);
    const auto sa = la.next();
    const auto sb = lb.next();
    auto loads = [&](auto first, auto mc) {
      constexpr int m = decltype(first)::value * P + decltype(mc)::value;
      static_for<m * T::kLoads / (4 * P), (m + 1) * T::kLoads / (4 * P)>([&](auto jc) { load(sa, sb, jc, cur); });
    };
    step(std::integral_constant<int, 3>{}, nxt, [&](auto mc) { loads(std::integral_constant<int, 0>{}, mc); });
    static_for<0, 3>([&](auto kc) {
      step(kc, nxt, [&](auto mc) { loads(std::integral_constant<int, decltype(kc)::value + 1>{}, mc); });
    });
    cur = nxt;
  }
  if (KT > 0)
    static_for<0, P>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      acc.v[m / BN][m % BN] = mfma<2>(fb[1][m % BN], fa[1][m / BN], acc.v[m / BN][m % BN]);
    });
  sched_fence();
  wait_vmcnt<0>();
  wait_lgkmcnt<0>();
  barrier();
}

// The wave's part of the tile in fp32, 32 rows at a time staged through LDS
// (the wave's own part) and stored 16 bytes a lane; ADD: added to what is there.
template <int BM, int BN, bool ADD>
__device__ __forceinline__ void kept_store32(const CheckpointArgs& a, const MidAccum<BM, BN>& acc, int64_t m0, int64_t n0,
                                             int wave, int lane) {
  constexpr uint32_t kRowBytes = 128 * BN + 16;
  const uint32_t area = wave * 32 * kRowBytes;
  const uint32_t st = area + (lane & 31) * kRowBytes + 16 * (lane >> 5);
  constexpr int kLanes = 8 * BN, kRows = 64 / kLanes;  // lanes a row, rows an access
  const int sub = lane / kLanes, chunk = lane % kLanes;
  const int64_t left = a.cols - n0 - 4 * chunk;
#pragma unroll
  for (int bi = 0; bi < BM; ++bi) {
    compiler_fence();
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& v = acc.v[bi][bj];
        *(MIGEMM_LDS f32x4*)lds_at(st + bj * 128 + q * 32) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    compiler_fence();
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
      const int64_t row = m0 + 32 * bi + kRows * i + sub;
      f32x4 v = *(const MIGEMM_LDS f32x4*)lds_at(area + (kRows * i + sub) * kRowBytes + chunk * 16);
      if (row < a.out_cols && left > 0) {
        float* d = static_cast<float*>(a.dw) + row * a.dw_rs + n0 + 4 * chunk;
        if (left >= 4) {
          if constexpr (ADD) v += *reinterpret_cast<const f32x4*>(d);
          *reinterpret_cast<f32x4*>(d) = v;
        } else {
          for (int e = 0; e < (int)left; ++e) d[e] = ADD ? d[e] + v[e] : v[e];
        }
      }
    }
  }
}

}  // namespace migemm
