// The kernels of attention over the 4-bit cache at head_dim 128.
#include "kv4_attn.cuh"

namespace cpattn {
namespace kvattn {
template cp_status run4_d<128>(const Params&, const Plan&, int64_t, int, cudaStream_t);
}  // namespace kvattn
}  // namespace cpattn
