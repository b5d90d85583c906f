// addbwd_bf16.cu -- the residual-stream backwards for bf16 activations.
#include "addbwd.cuh"

namespace gbn {

cudaError_t launch_add_bwd_bf16(cudaStream_t st, int mode, const BwdArgs& a, const RowPlan& p)
{
    return bwd_launch<__nv_bfloat16>(st, mode, a, p);
}

}  // namespace gbn
