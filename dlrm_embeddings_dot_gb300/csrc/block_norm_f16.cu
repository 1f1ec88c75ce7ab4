// block_norm_f16.cu -- the norms' kernels for fp16 rows.
#include "block_norm.cuh"

namespace dlrm {
namespace norms {

template dlrm_status forward<__half>(const NormFwd&, bool, cudaStream_t);
template dlrm_status backward<__half>(const NormBwd&, bool, cudaStream_t);

}  // namespace norms
}  // namespace dlrm
