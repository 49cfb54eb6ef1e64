// attn_prefix_rows_suffix_f16.cu - the few-row suffix stage for F16 (prefix_rows.cuh).
#include "prefix_rows.cuh"

namespace attn {
namespace prefix {
namespace rows {
template cudaError_t launch_suffix<false>(const Params&, int, bool, cudaStream_t);
template cudaError_t launch_join<false>(const Params&, cudaStream_t);
}  // namespace rows
}  // namespace prefix
}  // namespace attn
