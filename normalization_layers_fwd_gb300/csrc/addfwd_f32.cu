// addfwd_f32.cu -- the residual-stream forwards for f32 activations.
#include "addfwd.cuh"

namespace gbn {

cudaError_t launch_add_fwd_f32(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p)
{
    return fwd_launch<float>(st, mode, a, p);
}

}  // namespace gbn
