// attn_kv8_decode_e4m3.cu - e4m3 instances of attention over an 8-bit cache for few
// rows (attn_kv8_decode.cuh).
#include "attn_kv8_decode.cuh"

namespace attn {
namespace kv8 {

template cudaError_t launch_decode<FMT_E4M3>(const FwdParams& p, const DecodePlan& plan, cudaStream_t st);

}  // namespace kv8
}  // namespace attn
