// block_prefix.cu -- the route of a chunk over the block-scaled cache, and its workspace.
#include "block_prefix.cuh"

namespace i8kv {

cudaError_t launch_block_prefix_64(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_128(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_256(const bp::Params& pp, cudaStream_t stream);

namespace {

// Up to this many (token, head) rows of a KV head the chunk runs in groups of
// eight rows, each reading the int8 cache itself.
constexpr int kFewRows = 64;

int grid_of(const bp::Plan& w, int Hkv) {
  const int64_t most = (int64_t)w.nrb * w.ntiles * Hkv;
  const int sms = block_device_sms();
  return most < sms ? (int)most : sms;
}

}  // namespace

size_t block_prefix_workspace_bytes(int H, int C, int G, int Hkv, int D) {
  const int64_t rows = (int64_t)C * G;
  if (rows <= kFewRows)
    return block_decode_workspace_bytes(D, block_decode_grid((int)((rows + 7) / 8), Hkv, (H + C + 15) / 16));
  // without a window: the largest plan
  return bp::plan_of(H, C, G, Hkv, D, 0, block_device_sms()).bytes;
}

cudaError_t launch_block_prefix(BlockDecodeParams p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.C * p.G;
  if (rows <= kFewRows) {
    p.B = (int)((rows + 7) / 8);
    p.HG = 1;
    p.HH = p.Hkv;
    p.max_blocks = (p.H + p.C + 15) / 16;
    p.grid = block_decode_grid(p.B, p.HH, p.max_blocks);
    p.divGrid = FastDiv((uint32_t)p.grid);
    return launch_block_chunk_rows(p, stream);
  }
  bp::Params pp{p, bp::plan_of(p.H, p.C, p.G, p.Hkv, p.D, p.window, 1)};
  const int grid = grid_of(pp.w, p.Hkv);
  pp.w = bp::plan_of(p.H, p.C, p.G, p.Hkv, p.D, p.window, grid);
  pp.a.divGrid = FastDiv((uint32_t)grid);
  if (p.D == 256) return launch_block_prefix_256(pp, stream);
  if (p.D == 128) return launch_block_prefix_128(pp, stream);
  return launch_block_prefix_64(pp, stream);
}

}  // namespace i8kv
