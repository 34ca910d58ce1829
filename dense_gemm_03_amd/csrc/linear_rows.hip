// The kernels for few rows, of both input types.
#include "linear_configs.hpp"

namespace dg {

template <bool BF16, int FORM, int W, int WV>
hipError_t launch_few_rows(const LinearArgs &args, int blocks, hipStream_t stream)
{
    hipLaunchKernelGGL((few_rows_kernel<BF16, FORM, W, WV>), dim3(blocks), dim3(64 * WV), 0, stream, args);
    return hipGetLastError();
}

}  // namespace dg

#define DG_LIN_ROWS_INST(NAME, BF16, F, W, WV)                                             \
    template hipError_t dg::launch_few_rows<BF16, DG_LIN_FORM_ID_##F, W, WV>(              \
        const dg::LinearArgs &, int, hipStream_t);

DG_LIN_F32_ROWS(DG_LIN_ROWS_INST)
DG_LIN_BF16_ROWS(DG_LIN_ROWS_INST)
