// attn_kv8_decode_f16.cu - F16 instances of attention over an 8-bit cache for
// few rows (attn_kv8_decode.cuh).
#include "attn_kv8_decode.cuh"

namespace attn {
namespace kv8 {

template cudaError_t launch_decode<false>(const FwdParams& p, int fmt, cudaStream_t st);

}  // namespace kv8
}  // namespace attn
