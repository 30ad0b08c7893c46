// scaled_kernels.hip -- the product of 8-bit rows with a scale per row and
// per output channel:
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k])
// a and b are e4m3 codes, K-contiguous; the sum is fp32.
//
// scaled_tile: 256 x 256 or 192 x 256 tiles with the GEMM's K loop, where the
// product fills the chip with them (bound by the matrix instructions and the
// power they take: 8192 x 8192 x 16384 in 786 us, 2.80 PFLOP/s; 4000 x 3000 x
// 5000 in 62 us with 192 rows a tile, 252 tiles for 256 compute units, against
// 66 with 256 rows, 192 tiles).  scaled_mid: smaller tiles, their K split
// where there are few (bound by loads into LDS; 40 x 16384 x 8192 in 33 us,
// 4.1 TB/s of weights).  scaled_rows: tiles of 16 to 64 rows whose waves split
// K (bound by reading the weights, or by latency; 1 x 8192 x 8192 in 12.6 us,
// 5.3 TB/s).
#include "scaled_tiles.hpp"

namespace migemm {
namespace {

// The kernels (Variant), with figures for their cost.  128 x 128 comes
// twice: a ring of four slots, one workgroup a compute unit, hides the loads'
// latency where there is one tile a unit (424 x 6578 x 7971: 51 us, 58 with
// two slots); two slots, two workgroups a unit, each loading while the other
// multiplies, where there are more (1600 x 4000 x 16000: 125 us, 149 with 192
// rows a tile, 165 with 64 x 128; 2773 x 2191 x 552: 15.0, 25.6 and 18.4).
enum { kMidLast = 9, kExactRows, kExactMid };
const Variant kVariants[] = {
    tile_variant<kMulNative, 4>(1.1, 7.0),
    tile_variant<kMulNative, 3>(0.95, 6.0),
    rows_variant<1, 1, 1, 16, 2>(1),
    rows_variant<1, 1, 2, 16, 1>(2),
    rows_variant<1, 2, 2, 8, 1>(2),
    rows_variant<1, 4, 2, 8, 1>(2),
    mid_variant<kMulNative, 64, 64, 4>(2, 0.30, 0.48, 1.7),
    mid_variant<kMulNative, 64, 128, 3>(2, 0.43, 0.64, 1.3),
    mid_variant<kMulNative, 128, 128, 4>(1, 0.52, 0.52, 2.4),
    mid_variant<kMulNative, 128, 128, 2>(2, 0.60, 0.80, 2.0),
    rows_variant<kExactE4M3, 1, 4, 2, 1>(2),
    mid_variant<kMulExact, 64, 64, 2>(2, 0, 0, 0),
};
const CostModel kCost = {kMidLast, 5.5e6, 0.26, 0.6, false, 4.0, 5.2e6};

}  // namespace

// The kernel that costs least: the figures are a fit to 690 products of 1 to
// 8192 rows, 64 to 8192 columns and K of 257 to 16384, each timed with every
// kernel and up to 16 splits; what it picks is 2.5% slower than the fastest
// of them on average.
ScaledChoice choose_scaled(int64_t M, int64_t N, int64_t K, int cu_count) {
  // Short sums in exact products (rowblock.hpp): up to here fp32's own bound, K
  // 2^-23 of the sum of magnitudes, is about what the e4m3 instructions lose of
  // normal values, 1e-5 and at most 3e-5 of it.  Few results pay nothing for it
  // (300 x 2000 x 128: 4.9 us, 4.8 in e4m3; 16 x 8192 x 256: 4.5 and 4.7), many
  // up to twice the time (2000 x 4096 x 256: 15.6 and 8.3; 8192 x 8192 x 256: 85
  // and 44).  Further up it would be two to three times (16 x 8192 x 4096: 15.8
  // and 9.4; 2000 x 4096 x 1024: 31.5 and 13.5), where longer sums average the
  // loss out.
  if (K <= 256) return {M <= 16 ? kExactRows : kExactMid, 1, kTileM, 0};
  return cheapest_variant(kCost, kVariants, M, N, K, cu_count);
}

ScaledKernel scaled_kernel(int variant) {
  const Variant& v = kVariants[variant];
  return {v.tm, v.tn, lds_stages(kVariants, variant), variant >= kExactRows};
}

hipError_t prepare_scaled() { return prepare_variants(kVariants); }

hipError_t launch_scaled(const ScaledArgs& s, int variant, int cu_count, hipStream_t stream) {
  return launch_variant(kVariants[variant], variant <= kTile192, s, cu_count, stream);
}

}  // namespace migemm
