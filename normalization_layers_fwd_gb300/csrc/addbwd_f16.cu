// addbwd_f16.cu -- the residual-stream backwards for f16 activations.
#include "addbwd.cuh"

namespace gbn {

cudaError_t launch_add_bwd_f16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p)
{
    return bwd_launch<__half>(st, mode, a, p);
}

}  // namespace gbn
