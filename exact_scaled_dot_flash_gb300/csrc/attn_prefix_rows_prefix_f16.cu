// attn_prefix_rows_prefix_f16.cu - the few-row prefix stage for F16 (prefix_rows.cuh).
#include "prefix_rows.cuh"

namespace attn {
namespace prefix {
namespace rows {
template cudaError_t launch_prefix<false>(const Params&, int, cudaStream_t);
}  // namespace rows
}  // namespace prefix
}  // namespace attn
