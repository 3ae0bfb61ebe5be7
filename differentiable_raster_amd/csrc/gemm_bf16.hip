// The matrix products of the neural decoder for operands in bf16.
#include "gemm.h"

namespace gsmi {

hipError_t launch_gemm_bf16(TileShape shape, Layout la, Layout lb, EpiKind kind, const GemmArgs& g, hipStream_t s) {
    return gemm::launch_type<gemm::TBf16>(shape, la, lb, kind, g, s);
}
hipError_t launch_few_rows_bf16(EpiKind kind, const GemmArgs& g, hipStream_t s) {
    return gemm::launch_few_type<gemm::TBf16>(kind, g, s);
}
hipError_t launch_gradients_bf16(TileShape sx, TileShape sw, const GemmArgs& x, const GemmArgs& w, const ShareSum& c, hipStream_t s) {
    return gemm::launch_gradients_type<gemm::TBf16>(sx, sw, x, w, c, s);
}

}  // namespace gsmi
