// addbwd_f32.cu -- the residual-stream backwards for f32 activations.
#include "addbwd.cuh"

namespace gbn {

cudaError_t launch_add_bwd_f32(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p)
{
    return bwd_launch<float>(st, mode, a, p);
}

}  // namespace gbn
