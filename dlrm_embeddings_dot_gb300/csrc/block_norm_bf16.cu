// block_norm_bf16.cu -- the norms' kernels for bf16 rows.
#include "block_norm.cuh"

namespace dlrm {
namespace norms {

template dlrm_status forward<bf16>(const NormFwd&, bool, cudaStream_t);
template dlrm_status backward<bf16>(const NormBwd&, bool, cudaStream_t);

}  // namespace norms
}  // namespace dlrm
