// The kernels of attention over the 8-bit cache at head_dim 64.
#include "kv_attn.cuh"

namespace cpattn {
namespace kvattn {
template cp_status run_d<64>(const Params&, const Plan&, const CUtensorMap&, const CUtensorMap&, int64_t, int,
                             cudaStream_t);
}  // namespace kvattn
}  // namespace cpattn
