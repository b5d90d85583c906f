// addfwd_f16.cu -- the residual-stream forwards for f16 activations.
#include "addfwd.cuh"

namespace gbn {

cudaError_t launch_add_fwd_f16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p)
{
    return fwd_launch<__half>(st, mode, a, p);
}

}  // namespace gbn
