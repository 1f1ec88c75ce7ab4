// thin_grad8.cu -- the gradient of a dense layer of up to 16 outputs whose input and pre-activation are
// kept in 8 bits: the kernels of thin_grad.cuh, which read the bytes themselves.
#include "thin_grad.cuh"

namespace dlrm {
namespace thin {

dlrm_status run8(dlrm_dtype dt, const Grad& a, float* ws, cudaStream_t st)
{
    return with_type(dt, [&](auto t) { return run<decltype(t), true>(dt, a, ws, st); });
}

}  // namespace thin
}  // namespace dlrm
