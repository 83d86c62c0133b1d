// The product on CTA pairs in whole tiles (block128_pair.cuh).
#include "block128_pair.cuh"

namespace fp8g {

cudaError_t launch_b128_pair(const CUtensorMap &A, const CUtensorMap &B, const B128Params &p,
                             int out, bool vec_b, cudaStream_t stream) {
    const int grid = 2 * p.pairs;
    if (out == kB128Gated + FP8G_GATE_SILU)
        return launch_pair<false, kB128Gated + FP8G_GATE_SILU, false>(A, B, p, grid, stream);
    if (out == kB128Gated + FP8G_GATE_GELU)
        return launch_pair<false, kB128Gated + FP8G_GATE_GELU, false>(A, B, p, grid, stream);
    if (out == kB128Gated + FP8G_GATE_RELU)
        return launch_pair<false, kB128Gated + FP8G_GATE_RELU, false>(A, B, p, grid, stream);
    return vec_b ? launch_product<true, false>(A, B, p, out, grid, stream)
                 : launch_product<false, false>(A, B, p, out, grid, stream);
}

}  // namespace fp8g
