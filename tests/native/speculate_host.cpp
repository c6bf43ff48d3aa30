// The host side of the operators for speculative decoding (moe_speculate.cu), beside the
// layer operators', over the same runtime that only takes notes.
#include "layer_host.cpp"

#include "moe_speculate.cu"

namespace moe {

MOE_FAKE_LAUNCH(launch_kv_compact, const CompactParams &, cudaStream_t)
MOE_FAKE_LAUNCH(launch_kv_fork, const ForkParams &, cudaStream_t)
MOE_FAKE_LAUNCH(launch_sample, const moe_sample_desc &, int, cudaStream_t)

}  // namespace moe
