// The product on CTA pairs in whole tiles (block128_pair.cuh).  Where tiles scale B, ptxas spills one
// register (4 bytes out, 4 in), and the K blocks still take the MMAs' 725 cycles.
#include "block128_pair.cuh"

namespace fp8g {

cudaError_t launch_b128_pair(const B128Maps &m, const B128Params &p, int out, bool vec_b, cudaStream_t stream) {
    const int grid = 2 * p.pairs;
    if (out == kB128Gated + FP8G_GATE_SILU)
        return launch_pair<false, kB128Gated + FP8G_GATE_SILU, false>(m, p, grid, stream);
    if (out == kB128Gated + FP8G_GATE_GELU)
        return launch_pair<false, kB128Gated + FP8G_GATE_GELU, false>(m, p, grid, stream);
    if (out == kB128Gated + FP8G_GATE_RELU)
        return launch_pair<false, kB128Gated + FP8G_GATE_RELU, false>(m, p, grid, stream);
    return vec_b ? launch_product<true, false>(m, p, out, grid, stream)
                 : launch_product<false, false>(m, p, out, grid, stream);
}

}  // namespace fp8g
