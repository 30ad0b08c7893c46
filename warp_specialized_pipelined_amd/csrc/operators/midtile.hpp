// midtile.hpp -- output tiles smaller than 256 x 256, for products with too
// few large tiles to fill the chip, or too little K to pay for one.
//
// A workgroup of 4 waves takes a TM x TN tile, each wave a TM/2 x TN/2 quarter
// in blocks of 32 x 32.  The stages, their swizzles and the fragment layouts
// are those of the 256 x 256 K loop (kernel/mainloop.hpp): 128 bytes of K of
// each operand row, loaded straight into LDS.  What differs is that a small
// tile's stage is worth only 128 or 512 cycles of matrix instructions, less
// than a load takes to arrive and little more than an LDS read and a barrier
// do.  Two schedules:
//   SLOTS > 2, for few tiles with much K: the ring has SLOTS stages, all of
//     them in flight or waiting while one more, the stage being multiplied, is
//     wholly in registers: an iteration reads stage d + 1's fragments and
//     issues stage d + SLOTS's loads under the products of stage d, and meets
//     one barrier.
//   SLOTS = 2, for many tiles with little K: fragments one k-step ahead, as
//     in the 256 x 256 loop, in half the registers and half the LDS, so that
//     two 128 x 128 workgroups share a compute unit and one's loads arrive
//     under the other's products, prologue and epilogue.
//
// Bound: the loads.  A compute unit's L1 takes 31 cycles for 1 KiB of them
// (17 of address work, 14 stalled on lines on their way; counters over
// 2048 x 2048 x 16384 e4m3 in 128 x 128 tiles), so a 128 x 128 tile's stage of
// 32 KiB takes 1000 to 1200 cycles, 0.53 us measured, against 512 of matrix
// instructions; a 256 x 256 tile's takes 2000 against 2048.  Eight waves
// instead of four, more slots, padded rows and other cache policies change
// nothing.  So small tiles win only where large ones leave compute units idle
// or compute rows and columns that do not exist.
#pragma once

#include "../kernel/gfx950.hpp"
#include "../kernel/mainloop.hpp"
#include "../kernel/params.hpp"
#include "operators.h"
#include "rowblock.hpp"

namespace migemm {

// One operand's share of a stage: this wave's NL loads of 1 KiB (8 rows of 128
// bytes of K); load j of the wave fills LDS kilobyte NL wave + j of the
// operand's part of the slot.
template <int ES, bool KMAJ, int NL>
struct MidLoader {
  typedef StageGeom<ES> G;
  static_assert(NL == 1 || NL == 2 || NL == 4 || NL == 8, "a panel's loads come in whole shares");
  static_assert(KMAJ || ES == 2, "MN-contiguous operands are bf16");
  uint64_t at;         // address of (row 0 of the tile, the next stage's first k)
  int64_t kstep_bytes;  // from one stage to the next
  int64_t left;        // operand bytes from `at` to its end, rounded up to 16 (StageLoader::stage_rsrc)
  int krem;            // valid K from `at` on (capped: only "less than a stage" matters)
  uint32_t off[NL];
  int32_t kq[2];  // K index the lane's load j starts at, by the parity of j (K-contiguous) or at j = 0

  __device__ __forceinline__ int32_t kpos(int j) const { return KMAJ ? kq[j & 1] : kq[0] + 8 * j; }

  __device__ __forceinline__ void init(const void* ptr, int64_t bytes, int64_t ld, int64_t origin, int k0,
                                       int64_t K, int wave, int lane) {
    const int64_t first = KMAJ ? origin * ld * ES : origin * ES;
    kstep_bytes = KMAJ ? kStageKBytes : (int64_t)G::kK * ld * ES;
    at = reinterpret_cast<uint64_t>(ptr) + first + k0 * kstep_bytes;
    left = (bytes - first - k0 * kstep_bytes + 15) & ~(int64_t)15;
    const int64_t rem = K - (int64_t)k0 * G::kK;
    krem = rem > 0x7FFFFFFF ? 0x7FFFFFFF : (int)rem;
    if constexpr (KMAJ) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int row = (wave * NL + j) * 8 + (lane >> 3);
        off[j] = (uint32_t)(row * ld * ES) + (uint32_t)(((lane & 7) ^ swz_k8(row)) * 16);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)  // (swz_k8 of load j's row)
        kq[j] = ((lane & 7) ^ (4 * ((wave * NL + j) & 1) + (lane >> 4))) * G::kElemsPerChunk;
    } else {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int idx = wave * NL + j;
        const int krow = (idx % G::kLoadsPerPanel) * 8 + (lane >> 3);
        const int col = (idx / G::kLoadsPerPanel) * G::kPanelCols +
                        ((lane & 7) ^ swz_mn<ES>(krow)) * G::kElemsPerChunk;
        off[j] = (uint32_t)(krow * ld * ES) + (uint32_t)(col * ES);
      }
      kq[0] = 8 * ((wave * NL) % G::kLoadsPerPanel) + (lane >> 3);
      kq[1] = 0;
    }
  }
  // The next stage's resource and valid K; moves on to the one after it.
  struct Stage {
    __amdgpu_buffer_rsrc_t rsrc;
    int krem;
  };
  __device__ __forceinline__ Stage next() {
    const uint32_t bytes = left < 0 ? 0 : (left > 0x7FFFFFF0 ? 0x7FFFFFF0u : (uint32_t)left);
    const Stage s = {make_rsrc(reinterpret_cast<const void*>(at), bytes), krem};
    at += kstep_bytes;
    left -= kstep_bytes;
    krem -= G::kK;
    return s;
  }
  // Load j of the stage into the slot part at LDS offset `slot`; what lies
  // past K (or past the operand) reads as zero.
  __device__ __forceinline__ void load(const Stage& s, uint32_t slot, int wave, int j) const {
    dma16(s.rsrc, lds_at(slot + (wave * NL + j) * 1024), kpos(j) < s.krem ? off[j] : kOobOffset);
  }
  // Bytes past K in the chunks of a stage this wave loaded (StageLoader::clear_k_tail).
  __device__ __forceinline__ void clear_k_tail(uint32_t slot, int krem, int wave, int lane) const {
    if constexpr (KMAJ) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int nb = (krem - kpos(j)) * ES;
        if (nb > 0 && nb < 16) {
          MIGEMM_LDS u32x4* p = (MIGEMM_LDS u32x4*)lds_at(slot + (wave * NL + j) * 1024 + 16 * lane);
          u32x4 x = *p;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int vb = nb - 4 * w;
            x[w] &= vb >= 4 ? 0xFFFFFFFFu : (vb <= 0 ? 0u : (1u << (8 * vb)) - 1u);
          }
          *p = x;
        }
      }
    }
  }
};

// Fragment reads: K-contiguous ones are FragReader's; MN-contiguous ones as
// FragReader<2, false, 3>'s, a lane offset per block, since a wave's columns
// may start in the middle of a 64-column panel.
template <int ES, bool KMAJ, int NB>
struct MidReader;
template <int NB>
struct MidReader<2, true, NB> : FragReader<2, true, NB> {};
template <int NB>
struct MidReader<1, true, NB> : FragReader<1, true> {};
template <int NB>
struct MidReader<2, false, NB> {
  typedef StageGeom<2> G;
  uint32_t off[NB];
  __device__ __forceinline__ void init(int col0, int lane) {
    const int g = lane >> 4, t = lane & 15;
    const int k = 8 * (g >> 1) + (t >> 2);
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
    constexpr uint32_t c = 16 * KS * kPanelRowBytes;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MIGEMM_LDS i16x4*)lds_at(opnd + off[BLK] + c));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (MIGEMM_LDS i16x4*)lds_at(opnd + off[BLK] + c + 4 * kPanelRowBytes));
    const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
  }
};

// e4m3 fragments multiplied through bf16 (rowblock.hpp says why): 32 bytes a
// lane are four bf16 fragments.  Which K a register stands for does not
// matter, as both operands use the same order.
struct WideFrag {
  bf16x8 v[4];
};
__device__ __forceinline__ WideFrag widen_frag(i32x8 f) {
  WideFrag w;
  i32x4 lo, hi;
  widen(i32x4{f[0], f[1], f[2], f[3]}, lo, hi);
  w.v[0] = __builtin_bit_cast(bf16x8, lo);
  w.v[1] = __builtin_bit_cast(bf16x8, hi);
  widen(i32x4{f[4], f[5], f[6], f[7]}, lo, hi);
  w.v[2] = __builtin_bit_cast(bf16x8, lo);
  w.v[3] = __builtin_bit_cast(bf16x8, hi);
  return w;
}

// Geometry of a TM x TN tile.
template <int TM, int TN, int SLOTS>
struct MidGeom {
  static constexpr int kBM = TM / 64, kBN = TN / 64;  // a wave's 32 x 32 blocks
  static constexpr uint32_t kPartA = TM * kStageKBytes, kSlot = (TM + TN) * kStageKBytes;
  static constexpr uint32_t kRing = SLOTS * kSlot;
  // Epilogue staging: a wave's 32 kBM rows of 32 kBN bf16 and 16 bytes of padding.
  static constexpr uint32_t kStaging = 4 * 32 * kBM * (64 * kBN + 16);
  static constexpr uint32_t kLds = kRing > kStaging ? kRing : kStaging;
};

// A wave's quarter of the tile, laid out as mainloop.hpp's Accum.
template <int BM, int BN>
struct MidAccum {
  f32x16 v[BM][BN];
};

// How bytes are multiplied: as e4m3 by its own instructions, through bf16
// (rowblock.hpp), or as int8 (sums: int32 bits).
enum MidMul { kMulNative, kMulExact, kMulInt8 };

// K stages [k0, k0 + KT) of the tile at (m0, n0); loads past kend (at most K)
// read as zero.  On return every wave is done with the ring.
template <int ES, bool AK, bool BK, int TM, int TN, int SLOTS, MidMul MUL = kMulNative>
__device__ __forceinline__ void mid_loop(MidAccum<TM / 64, TN / 64>& acc, const KernelArgs& a, int64_t m0,
                                         int64_t n0, int wave, int lane, int k0, int KT, int64_t kend) {
  typedef StageGeom<ES> G;
  typedef MidGeom<TM, TN, SLOTS> T;
  typedef typename FragType<ES>::type frag_t;
  constexpr int BM = T::kBM, BN = T::kBN, NLA = TM / 32, NLB = TN / 32;
  constexpr int kLoads = NLA + NLB;  // a wave's loads of a stage
  constexpr int KS = G::kKSteps;
  MidLoader<ES, AK, NLA> la;
  MidLoader<ES, BK, NLB> lb;
  la.init(a.A, a.a_bytes, a.lda, m0, k0, kend, wave, lane);
  lb.init(a.B, a.b_bytes, a.ldb, n0, k0, kend, wave, lane);
  MidReader<ES, AK, BM> ra;
  MidReader<ES, BK, BN> rb;
  ra.init((wave >> 1) * 32 * BM, lane);
  rb.init((wave & 1) * 32 * BN, lane);
#pragma unroll
  for (int i = 0; i < BM; ++i)
#pragma unroll
    for (int j = 0; j < BN; ++j) acc.v[i][j] = f32x16{};

  // Fragments: of two stages (the one being multiplied, the one being read),
  // or with two slots of two k-steps.
  constexpr bool kDeep = SLOTS > 2;
  constexpr int FS = kDeep ? KS : 1;
  frag_t fa[2][FS][BM], fb[2][FS][BN];
  constexpr int P = BM * BN, R = BM + BN;
  // Fragment x of k-step KSTEP (A's BM blocks, then B's BN) into buffer b, place f.
  auto read = [&](auto bc, auto fc, auto kc, auto xc, uint32_t slot) {
    constexpr int b = decltype(bc)::value, f = decltype(fc)::value, ks = decltype(kc)::value;
    constexpr int x = decltype(xc)::value;
    if constexpr (x < BM) fa[b][f][x] = ra.template read<x, ks>(slot);
    else fb[b][f][x - BM] = rb.template read<x - BM, ks>(slot + T::kPartA);
  };
  // Product m of the k-step in buffer b, place f.
  constexpr bool kExact = MUL == kMulExact;
  WideFrag wa[kExact ? BM : 1], wb[kExact ? BN : 1];
  auto multiply = [&](auto bc, auto fc, auto mc) {
    constexpr int b = decltype(bc)::value, f = decltype(fc)::value;
    constexpr int i = decltype(mc)::value / BN, j = decltype(mc)::value % BN;
    if constexpr (kExact) {
      if constexpr (i == 0 && j == 0) {
#pragma unroll
        for (int x = 0; x < BM; ++x) wa[x] = widen_frag(fa[b][f][x]);
#pragma unroll
        for (int x = 0; x < BN; ++x) wb[x] = widen_frag(fb[b][f][x]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) acc.v[i][j] = mfma<2>(wb[j].v[q], wa[i].v[q], acc.v[i][j]);
    } else if constexpr (MUL == kMulInt8) {
      acc.v[i][j] = mfma_i8_32x32x64(fb[b][f][j], fa[b][f][i], acc.v[i][j]);
    } else {
      acc.v[i][j] = mfma<ES>(fb[b][f][j], fa[b][f][i], acc.v[i][j]);
    }
  };
  // Load j of a stage: A's, then B's.
  auto load = [&](const auto& sa, const auto& sb, auto jc, uint32_t slot) {
    constexpr int j = decltype(jc)::value;
    if constexpr (j < NLA) la.load(sa, slot, wave, j);
    else lb.load(sb, slot + T::kPartA, wave, j - NLA);
  };
  // Relative stage rs, landed in `slot`: clear what lies past K in its chunks.
  auto clear_tail = [&](int rs, uint32_t slot) {
    if constexpr (AK || BK) {
      const int64_t krem = kend - (int64_t)(k0 + rs) * G::kK;
      if (krem > 0 && krem < G::kK && ((krem * ES) & 15) != 0) {
        la.clear_k_tail(slot, (int)krem, wave, lane);
        lb.clear_k_tail(slot + T::kPartA, (int)krem, wave, lane);
        wait_lgkmcnt<0>();
      }
    }
  };
  // Waits until all but the last `ahead` (at most SLOTS - 1) stages' loads have landed.
  auto landed = [&](int ahead) {
    sched_fence();
    static_for<0, SLOTS>([&](auto ac) {
      constexpr int n = decltype(ac)::value;
      if (ahead == n) wait_vmcnt<kLoads * n>();
    });
    sched_fence();
  };
  auto after = [](uint32_t slot) { return slot + T::kSlot == T::kRing ? 0 : slot + T::kSlot; };
  const std::integral_constant<int, 0> zero;

  static_for<0, SLOTS>([&](auto sc) {
    if (decltype(sc)::value < KT) {
      const auto sa = la.next();
      const auto sb = lb.next();
      static_for<0, kLoads>([&](auto jc) { load(sa, sb, jc, decltype(sc)::value * T::kSlot); });
    }
  });
  if (KT > 0) {
    landed(KT - 1 < SLOTS - 1 ? KT - 1 : SLOTS - 1);
    clear_tail(0, 0);
    barrier();
  }
  uint32_t cur = 0;
  if constexpr (kDeep) {
    // Stage d from buffer b; stage d + 1 (in slot `nxt`) into the other buffer;
    // stage d + SLOTS loaded into `cur`, which stage d's reads left free.  The
    // reads go first, one or two in front of each product, and the loads one
    // behind each product from the first on (the address path takes 16 cycles
    // a load and four waves share it: in a burst they stall what follows).
    auto stage = [&](auto bc, int d) {
      constexpr int b = decltype(bc)::value;
      const uint32_t nxt = after(cur);
      const bool more = d + SLOTS < KT;
      const auto sa = la.next();
      const auto sb = lb.next();
      static_for<0, KS * P>([&](auto mc) {
        constexpr int m = decltype(mc)::value;
        sched_fence();
        static_for<m * KS * R / (KS * P), (m + 1) * KS * R / (KS * P)>([&](auto xc) {
          constexpr int x = decltype(xc)::value;
          read(std::integral_constant<int, 1 - b>{}, std::integral_constant<int, x / R>{},
               std::integral_constant<int, x / R>{}, std::integral_constant<int, x % R>{}, nxt);
        });
        multiply(bc, std::integral_constant<int, m / P>{}, std::integral_constant<int, m % P>{});
        static_for<m * kLoads / (KS * P), (m + 1) * kLoads / (KS * P)>([&](auto jc) {
          if (more) load(sa, sb, jc, cur);
        });
      });
      // This wave's part of stage d + 2 has landed and its reads of stage d + 1
      // have returned; past the barrier that holds for every wave.
      const int ahead = KT - 3 - d;
      landed(ahead < 0 ? 0 : (ahead < SLOTS - 2 ? ahead : SLOTS - 2));
      wait_lgkmcnt<0>();
      clear_tail(d + 2, after(nxt));
      barrier();
      cur = nxt;
    };
    if (KT > 0) {
      static_for<0, KS * R>([&](auto xc) {
        constexpr int x = decltype(xc)::value;
        read(zero, std::integral_constant<int, x / R>{}, std::integral_constant<int, x / R>{},
             std::integral_constant<int, x % R>{}, 0);
      });
      landed(KT < 2 ? 0 : (KT - 2 < SLOTS - 2 ? KT - 2 : SLOTS - 2));
      wait_lgkmcnt<0>();
      clear_tail(1, T::kSlot);
      barrier();
    }
    for (int d = 0; d < KT; d += 2) {
      stage(std::integral_constant<int, 0>{}, d);
      if (d + 1 == KT) break;
      stage(std::integral_constant<int, 1>{}, d + 1);
    }
  } else {
    if (KT > 0) static_for<0, R>([&](auto xc) { read(zero, zero, zero, xc, 0); });
    for (int d = 0; d < KT; ++d) {
      const uint32_t nxt = after(cur);
      static_for<0, KS - 1>([&](auto kc) {
        constexpr int ks = decltype(kc)::value;
        static_for<0, P>([&](auto mc) {
          constexpr int m = decltype(mc)::value;
          sched_fence();
          static_for<m * R / P, (m + 1) * R / P>([&](auto xc) {
            read(std::integral_constant<int, (ks + 1) & 1>{}, zero, std::integral_constant<int, ks + 1>{}, xc, cur);
          });
          multiply(std::integral_constant<int, ks & 1>{}, zero, mc);
        });
      });
      // Stage d + 1 has landed and this wave's reads of stage d have returned;
      // past the barrier that holds for every wave, and stage d + 2 may be
      // loaded over stage d.
      landed(0);
      wait_lgkmcnt<0>();
      clear_tail(d + 1, nxt);
      barrier();
      const bool more = d + 2 < KT;
      const auto sa = la.next();
      const auto sb = lb.next();
      static_for<0, P>([&](auto mc) {
        constexpr int m = decltype(mc)::value;
        sched_fence();
        static_for<m * R / P, (m + 1) * R / P>([&](auto xc) { read(zero, zero, zero, xc, nxt); });
        multiply(std::integral_constant<int, (KS - 1) & 1>{}, zero, mc);
        static_for<m * kLoads / P, (m + 1) * kLoads / P>([&](auto jc) {
          if (more) load(sa, sb, jc, cur);
        });
      });
      cur = nxt;
    }
  }
  sched_fence();
  wait_vmcnt<0>();
  wait_lgkmcnt<0>();
  barrier();
}

// fp32 sums of a workgroup's tile in memory, in register order: 16-byte pieces
// [item][wave][block][q][lane].
template <int BM, int BN>
__device__ __forceinline__ void mid_put(mid_piece* sums, int64_t item, const MidAccum<BM, BN>& acc, int wave,
                                        int lane) {
  mid_piece* p = sums + ((item * 4 + wave) * BM * BN) * 256 + lane;
#pragma unroll
  for (int b = 0; b < BM * BN; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x16& v = acc.v[b / BN][b % BN];
      p[(4 * b + q) * 64] = mid_piece{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    }
}
// Adds such sums to acc.
template <int BM, int BN>
__device__ __forceinline__ void mid_add_all(const mid_piece* sums, int64_t item, MidAccum<BM, BN>& acc, int wave,
                                            int lane) {
  const mid_piece* p = sums + ((item * 4 + wave) * BM * BN) * 256 + lane;
#pragma unroll
  for (int b = 0; b < BM * BN; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const mid_piece x = p[(4 * b + q) * 64];
#pragma unroll
      for (int c = 0; c < 4; ++c) acc.v[b / BN][b % BN][4 * q + c] += x[c];
    }
}
// Adds one block of such sums to acc (INT: int32 bits, acc's too).
template <int BM, int BN, bool INT = false>
__device__ __forceinline__ void mid_add(const mid_piece* sums, int64_t item, MidAccum<1, 1>& acc, int wave,
                                        int block, int lane) {
  const mid_piece* p = sums + ((item * 4 + wave) * BM * BN + block) * 256 + lane;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const mid_piece x = p[64 * q];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float v = acc.v[0][0][4 * q + c];
      acc.v[0][0][4 * q + c] = INT ? __int_as_float(__float_as_int(v) + __float_as_int(x[c])) : v + x[c];
    }
  }
}
// Four results of a row, rounded to bf16, where `left` columns are left from
// d on (none, if it is not positive).
__device__ __forceinline__ void store4(unsigned short* d, int64_t left, f32x4 x) {
  const u32x2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
  if (left >= 4) {
    *reinterpret_cast<u32x2*>(d) = w;
  } else {
    for (int c = 0; c < (int)left; ++c) d[c] = (unsigned short)(w[c >> 1] >> (16 * (c & 1)));
  }
}

// Tile number `t` of tiles_m x tiles_n: down the columns in groups of 8 tile
// rows, so that consecutive numbers share operand panels.
struct MidTile {
  int tm, tn;
};
__device__ __forceinline__ MidTile mid_tile(int t, int tiles_m, int tiles_n) {
  const int g = t / (8 * tiles_n), r = t - g * 8 * tiles_n;
  const int rows = min(tiles_m - 8 * g, 8);
  return {8 * g + r % rows, r / rows};
}

// The wave's part of the tile, each value transformed, rounded to bf16,
// staged through LDS (the wave's own part) and stored 16 bytes a lane.
// value(bi, bj, q): the four results of row 32 bi + l % 32, columns
// 32 bj + 8 q + 4 (l / 32) .. + 3 of the part, which starts at (m0, n0);
// row_of(r): the row of D that row r goes to, for rows below M.
template <int BM, int BN, class Value, class RowOf>
__device__ __forceinline__ void mid_store(void* D, int64_t ldd, int64_t M, int64_t N, int64_t m0, int64_t n0,
                                          int wave, int lane, Value&& value, RowOf&& row_of) {
  constexpr uint32_t kRowBytes = 64 * BN + 16;
  const uint32_t area = wave * 32 * BM * kRowBytes;
  const uint32_t st = area + (lane & 31) * kRowBytes + 8 * (lane >> 5);
#pragma unroll
  for (int bi = 0; bi < BM; ++bi)
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = value(bi, bj, q);
        const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *(MIGEMM_LDS u32x2*)lds_at(st + 32 * bi * kRowBytes + (4 * bj + q) * 16) = w;
      }
  constexpr int kLanes = 4 * BN, kRows = 64 / kLanes;  // lanes a row, rows an access
  const int sub = lane / kLanes, chunk = lane % kLanes;
  const int64_t cols_left = N - n0 - 8 * chunk;
#pragma unroll
  for (int i = 0; i < 32 * BM / kRows; ++i) {
    const int row = kRows * i + sub;
    const u32x4 v = *(const MIGEMM_LDS u32x4*)lds_at(area + row * kRowBytes + chunk * 16);
    if (m0 + row < M && cols_left > 0) {
      unsigned short* d = static_cast<unsigned short*>(D) + row_of(m0 + row) * ldd + n0 + 8 * chunk;
      if (cols_left >= 8) {
        *reinterpret_cast<u32x4*>(d) = v;
      } else {
        for (int e = 0; e < (int)cols_left; ++e) d[e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

}  // namespace migemm
