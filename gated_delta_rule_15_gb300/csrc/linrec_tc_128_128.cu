// linrec_tc_128_128.cu -- linrec_tc.cuh's kernel for key width 128, value width 128.
#include "linrec_tc.cuh"

namespace dr {
namespace linrec {
int launch_128_128(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s) {
    return dot ? launch<128, 128, true>(maps, a, grid, s) : launch<128, 128, false>(maps, a, grid, s);
}
}  // namespace linrec
}  // namespace dr
