// addfwd_bf16.cu -- the residual-stream forwards for bf16 activations.
#include "addfwd.cuh"

namespace gbn {

cudaError_t launch_add_fwd_bf16(cudaStream_t st, int mode, const FwdArgs& a, const RowPlan& p)
{
    return fwd_launch<__nv_bfloat16>(st, mode, a, p);
}

}  // namespace gbn
