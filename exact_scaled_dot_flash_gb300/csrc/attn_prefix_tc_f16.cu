// attn_prefix_tc_f16.cu - both stages of a shared prefix for many rows, F16 (prefix_tc.cuh).
#include "prefix_tc.cuh"

namespace attn {
namespace prefix {
namespace tc {
template cudaError_t launch<false, true>(EncodeTiledFn, const Params&, bool, cudaStream_t);
template cudaError_t launch<false, false>(EncodeTiledFn, const Params&, bool, cudaStream_t);
}  // namespace tc
}  // namespace prefix
}  // namespace attn
