// block_norm_f32.cu -- the norms' kernels for fp32 rows.
#include "block_norm.cuh"

namespace dlrm {
namespace norms {

template dlrm_status forward<float>(const NormFwd&, bool, cudaStream_t);
template dlrm_status backward<float>(const NormBwd&, bool, cudaStream_t);

}  // namespace norms
}  // namespace dlrm
