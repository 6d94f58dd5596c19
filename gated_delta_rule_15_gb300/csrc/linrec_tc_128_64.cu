// linrec_tc_128_64.cu -- linrec_tc.cuh's kernel for key width 128, value width 64.
#include "linrec_tc.cuh"

namespace dr {
namespace linrec {
int launch_128_64(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s) {
    return dot ? launch<128, 64, true>(maps, a, grid, s) : launch<128, 64, false>(maps, a, grid, s);
}
}  // namespace linrec
}  // namespace dr
