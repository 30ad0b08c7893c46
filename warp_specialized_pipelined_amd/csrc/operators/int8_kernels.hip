// int8_kernels.hip -- the product of int8 rows with a scale per row and per
// output channel, and a bias per channel:
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k] + bias[n])
// The sum is int32 and exact (K is at most 131071: 131071 * 128 * 128 < 2^31),
// so the order of the additions, K's split among them, does not matter.
//
// The kernels are the scaled product's (scaled_tiles.hpp), with two
// v_mfma_i32_32x32x32_i8 in place of one 32x32x64 e4m3 instruction: the same
// bytes of K a lane, the same fragments, the same cycles.
#include "scaled_tiles.hpp"

namespace migemm {
namespace {

const Variant kVariants[] = {
    tile_variant<kMulInt8, 4>(1.1, 7.0),
    tile_variant<kMulInt8, 3>(0.95, 6.0),
    rows_variant<kInt8, 1, 1, 16, 2>(1),
    rows_variant<kInt8, 1, 2, 16, 1>(2),
    rows_variant<kInt8, 2, 2, 8, 1>(2),
    rows_variant<kInt8, 4, 2, 8, 1>(2),
    mid_variant<kMulInt8, 64, 64, 4>(2, 0.30, 0.48, 1.7),
    mid_variant<kMulInt8, 64, 128, 3>(2, 0.43, 0.64, 1.3),
    mid_variant<kMulInt8, 128, 128, 4>(1, 0.52, 0.52, 2.4),
    mid_variant<kMulInt8, 128, 128, 2>(2, 0.60, 0.80, 2.0),
};

}  // namespace

ScaledChoice choose_int8(int64_t M, int64_t N, int64_t K, int cu_count) {
  return cheapest_variant(kVariants, M, N, K, cu_count);
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
