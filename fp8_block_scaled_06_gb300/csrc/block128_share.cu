// The product on CTA pairs where pairs share the K blocks of tiles (block128_pair.cuh).
// Variants of their own: the bookkeeping in registers cost the whole-tile loop 5%.  ptxas spills two to
// four of these variants' registers (16 bytes out, 84 in at most).
#include "block128_pair.cuh"

namespace fp8g {

cudaError_t launch_b128_share(const B128Maps &m, const B128Params &p, int out, bool vec_b, cudaStream_t stream) {
    const int grid = 2 * p.pairs;
    return vec_b ? launch_product<true, true>(m, p, out, grid, stream)
                 : launch_product<false, true>(m, p, out, grid, stream);
}

}  // namespace fp8g
