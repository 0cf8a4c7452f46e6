// block_decode_wide.cu -- the decode attention of block_decode.cuh with 16 query
// rows per pass.
#include "block_decode.cuh"

namespace i8kv {
I8KV_DEFINE_ERROR_ACCESSOR(read_error_block_decode_wide)

cudaError_t launch_block_rows_wide(const BlockDecodeParams& p, bool chunk, cudaStream_t stream) {
  return launch_rows<16>(p, chunk, stream);
}
}  // namespace i8kv
