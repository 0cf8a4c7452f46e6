// block_prefix_64.cu -- the chunk attention of block_prefix.cuh at head_dim 64.
#include "block_prefix.cuh"

namespace i8kv {
I8KV_DEFINE_ERROR_ACCESSOR(read_error_block_prefix_64)

cudaError_t launch_block_prefix_64(const bp::Params& pp, cudaStream_t stream) { return bp::launch_any<64>(pp, stream); }
}  // namespace i8kv
