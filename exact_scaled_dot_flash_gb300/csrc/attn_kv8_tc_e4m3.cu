// attn_kv8_tc_e4m3.cu - e4m3 instances of attention over an 8-bit cache for many
// rows (attn_kv8_tc.cuh).
#include "attn_kv8_tc.cuh"

namespace attn {
namespace kv8 {

template cudaError_t launch_tc<FMT_E4M3>(const FwdParams& p, cudaStream_t st);

}  // namespace kv8
}  // namespace attn
