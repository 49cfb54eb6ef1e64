// attn_prefix_rows_prefix_bf16.cu - the few-row prefix stage for BF16 (prefix_rows.cuh).
#include "prefix_rows.cuh"

namespace attn {
namespace prefix {
namespace rows {
template cudaError_t launch_prefix<true>(const Params&, int, cudaStream_t);
}  // namespace rows
}  // namespace prefix
}  // namespace attn
