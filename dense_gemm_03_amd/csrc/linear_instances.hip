// One slice of the linear-layer kernels: one input type and one form.  The
// build compiles this file once per slice, with DG_LIN_TABLE set to
// DG_LIN_F32_TABLE or DG_LIN_BF16_TABLE and DG_LIN_FORM to N, T or W (w as K x
// N, w as N x K, weight gradient).
#if !defined(DG_LIN_TABLE) || !defined(DG_LIN_FORM)
#error "define DG_LIN_TABLE and DG_LIN_FORM"
#endif
#include "linear_configs.hpp"

namespace dg {

template <bool BF16, int BM, int BN, int BK, int WM, int WN, int STAGES, int LX, int LW, bool ALIGNED>
hipError_t launch_linear(const LinearArgs &args, int blocks, hipStream_t stream)
{
    hipLaunchKernelGGL((linear_kernel<BF16, BM, BN, BK, WM, WN, STAGES, LX, LW, ALIGNED>),
                       dim3(blocks), dim3(64 * WM * WN), 0, stream, args);
    return hipGetLastError();
}

}  // namespace dg

#define DG_LIN_INST(BF16, BM, BN, BK, WM, WN, S, F)                                              \
    template hipError_t dg::launch_linear<BF16, BM, BN, BK, WM, WN, S, DG_LIN_LX_##F,            \
                                          DG_LIN_LW_##F, true>(const dg::LinearArgs &, int,      \
                                                               hipStream_t);                     \
    template hipError_t dg::launch_linear<BF16, BM, BN, BK, WM, WN, S, DG_LIN_LX_##F,            \
                                          DG_LIN_LW_##F, false>(const dg::LinearArgs &, int,     \
                                                                hipStream_t);
#define DG_LIN_INST_FORM2(BF16, BM, BN, BK, WM, WN, S, F) DG_LIN_INST(BF16, BM, BN, BK, WM, WN, S, F)
#define DG_LIN_INST_ENTRY(NAME, BF16, BM, BN, BK, WM, WN, S, GM, STEP, ALONE, BLOCK) \
    DG_LIN_INST_FORM2(BF16, BM, BN, BK, WM, WN, S, DG_LIN_FORM)

DG_LIN_TABLE(DG_LIN_INST_ENTRY)
