// attn_prefix_tc_bf16.cu - both stages of a shared prefix for many rows, BF16 (prefix_tc.cuh).
#include "prefix_tc.cuh"

namespace attn {
namespace prefix {
namespace tc {
template cudaError_t launch<true, true>(EncodeTiledFn, const Params&, bool, cudaStream_t);
template cudaError_t launch<true, false>(EncodeTiledFn, const Params&, bool, cudaStream_t);
}  // namespace tc
}  // namespace prefix
}  // namespace attn
