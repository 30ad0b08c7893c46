// int8_kernels.hip -- the product of int8 rows with a scale per row and per
// output channel, and a bias per channel:
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k] + bias[n])
// The sum is int32 and exact (K is at most 131071: 131071 * 128 * 128 < 2^31),
// so the order of the additions, K's split among them, does not matter.
//
// The kernels are the scaled product's (scaled_tiles.hpp), with two
// v_mfma_i32_32x32x32_i8 in place of one 32x32x64 e4m3 instruction: the same
// bytes of K a lane, the same fragments.  Few rows are bound by b's bytes. 1 x
// 8192 x 8192 takes 14.9 us with b from memory, 4.5 TB/s, and 12.3 with two b's
// in turn, which the 256 MB last-level cache holds; 33 x 16384 x 8192 33 us (4.1
// TB/s) and 27, and from memory 30 where b's stride is 8320: one of a power of
// two sends a stage's rows to few channels.  Many rows are bound by the matrix
// instructions (8192 x 8192 x 16384: 800 to 860 us from card to card, 2.6 to 2.7
// POP/s; 4000 x 3000 x 5000, one round of 252 tiles: 64 to 68 us).
#include "scaled_tiles.hpp"

namespace migemm {
namespace {

// The scaled product's tiles, but for a second 128 x 128 with four stages in
// LDS: it was the fastest of 6 of 2200 products, by up to 8% (71 x 15970 x
// 11880), and the cost below would not find those.
const Variant kVariants[] = {
    tile_variant<kMulInt8, 4>(1.03, 9.6),
    tile_variant<kMulInt8, 3>(0.78, 8.0),
    rows_variant<kInt8, 1, 1, 16, 2>(1, 67e3, 1.5),
    rows_variant<kInt8, 1, 2, 16, 1>(2, 49e3, 1.1),
    rows_variant<kInt8, 2, 2, 8, 1>(2, 55e3, 0.4),
    rows_variant<kInt8, 4, 2, 8, 1>(2, 47e3, 0.7),
    mid_variant<kMulInt8, 64, 64, 4>(2, 0.26, 0.47, 2.3),
    mid_variant<kMulInt8, 64, 128, 3>(2, 0.42, 0.44, 3.3),
    mid_variant<kMulInt8, 128, 128, 2>(2, 0.63, 0.63, 3.2),
};
constexpr int kLast = sizeof(kVariants) / sizeof(kVariants[0]) - 1;
const CostModel kCost = {kLast, 10.4e6, 0.25, 1.1, true, 7.5, 11e6};

}  // namespace

// The kernel that costs least: the figures are a fit to 2200 products, 1235 of
// 1 to 16384 rows, 64 to 16384 columns and K of 64 to 16384 and 965 of up to 200
// rows, 512 to 17000 columns and K of 512 to 16384, each timed with every kernel
// and up to 16 splits.  What it picks is 1.7% and 2.2% slower than the fastest
// of them on average (4.7% and 5.9% with the e4m3 product's figures).  Each was
// timed on two sets of operands in turn, so that operands of up to 128 MB came
// from the last-level cache, whose rate kCost's memory rate is (10.4 TB/s; a copy
// moves 5.2).  From memory what it picks takes 3 to 24% longer (33 x 8192 x 8192
// 19.3 and 21.1 us, 64 x 11008 x 4096 15.0 and 17.4, 300 x 2000 x 4096 15.0 and
// 15.6, 128 x 8192 x 8192 26.4 and 27.6); whether another kernel would then be
// the fastest was not measured.
ScaledChoice choose_int8(int64_t M, int64_t N, int64_t K, int cu_count) {
  return cheapest_variant(kCost, kVariants, M, N, K, cu_count);
}

ScaledKernel int8_kernel(int variant) {
  const Variant& v = kVariants[variant];
  return {v.tm, v.tn, lds_stages(kVariants, variant), false};
}

hipError_t prepare_int8() { return prepare_variants(kVariants); }

hipError_t launch_int8(const ScaledArgs& s, int variant, int cu_count, hipStream_t stream) {
  return launch_variant(kVariants[variant], variant <= kTile192, s, cu_count, stream);
}

}  // namespace migemm
