// The matrix products of the neural decoder for operands in e4m3.
#include "gemm.h"

namespace gsmi {

hipError_t launch_gemm_e4m3(TileShape shape, Layout la, Layout lb, EpiKind kind, const GemmArgs& g, hipStream_t s) {
    return gemm::launch_type<gemm::TE4m3>(shape, la, lb, kind, g, s);
}
hipError_t launch_few_rows_e4m3(EpiKind kind, const GemmArgs& g, hipStream_t s) {
    return gemm::launch_few_type<gemm::TE4m3>(kind, g, s);
}

}  // namespace gsmi
