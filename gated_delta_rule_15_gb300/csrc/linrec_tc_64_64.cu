// linrec_tc_64_64.cu -- linrec_tc.cuh's kernel for key width 64, value width 64.
#include "linrec_tc.cuh"

namespace dr {
namespace linrec {
int launch_64_64(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s) {
    return dot ? launch<64, 64, true>(maps, a, grid, s) : launch<64, 64, false>(maps, a, grid, s);
}
}  // namespace linrec
}  // namespace dr
