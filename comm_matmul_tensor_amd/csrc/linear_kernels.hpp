// Launches shared by the linear's translation units: the tiled product
// (gemm_linear_bf16.hip, gemm_linear_f16.hip) and the plan it follows.
#pragma once
#include "linear_gemm.hpp"

namespace mc2 {
namespace lin {

// The tiles: 256 x 256 in two LDS stages, 128 x 256 in three, 128 x 128 in
// four.  A larger tile reads less per product; a smaller one fills the CUs
// better, and its deeper ring of stages covers more of the latency.  The
// tiles under 128 x 128 (four stages) are for products of few tiles and for
// groups of few rows; those of 96 rows need a K-contiguous A.
enum Tile : int { TILE_256X256, TILE_128X256, TILE_128X128, TILE_96X128, TILE_128X64, TILE_96X64, TILE_64X64 };

// Tile and split of a product, from its sizes alone (the workspace's size
// follows it).
struct Plan {
  Tile tile;
  int splits;        // parts of K (dense, 128 columns or fewer), each k_part long
  int64_t k_part;
  size_t partial_bytes;
};
// Layout: 0 A K-, B K-contiguous (forward); 1 A K-, B N-contiguous (dx);
// 2 A M-, B N-contiguous (dw).
Plan plan_product(int64_t m, int64_t n, int64_t k, int layout, int gmode, int64_t groups);

// The product's splits, k_part, partial, order
// and epilogue are set here from the plan.
template <int DT>
hipError_t launch_product(const Product& p, int layout, int gmode, const Plan& plan, hipStream_t s);

}  // namespace lin
}  // namespace mc2
