// block_prefix.cu -- the route of a chunk over the block-scaled cache, and its workspace.
#include "block_prefix.cuh"

namespace i8kv {

cudaError_t launch_block_prefix_64(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_128(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_256(const bp::Params& pp, cudaStream_t stream);

namespace {

// Few (token, head) rows of a KV head run in groups of eight, each reading the
// int8 cache itself; more run in 128-row blocks on 16-bit operand tiles, which
// have to be made first.  With X = keys x Hkv x D in millions and g groups the
// first takes about 6 + 0.4 g X us and the second 13 + 3.2 X (measured: 24/4/256,
// 8192 keys, 60 rows 33 against 40 us, 126 rows 51 against 42; 1000 keys, 64 rows
// 9 against 21, 126 rows 12 against 22).  More (group, KV head) pairs than SMs
// pay for each pair's start and end instead (8/8/64, 64 keys, 192 rows: 34 against
// 15 us), so beyond 64 rows the pairs have to fit.
bool few_rows(int H, int C, int G, int Hkv, int D, int window) {
  const int64_t groups = ((int64_t)C * G + 7) / 8;
  const int64_t keys = window > 0 && (int64_t)window < H ? (int64_t)window + C : (int64_t)H + C;
  return groups <= 8 || (groups <= 24 && groups * Hkv <= 128 && (groups - 8) * keys * Hkv * D <= 16000000);
}

int grid_of(const bp::Plan& w, int Hkv) {
  const int64_t most = (int64_t)w.nrb * w.ntiles * Hkv;
  const int sms = block_device_sms();
  return most < sms ? (int)most : sms;
}

}  // namespace

size_t block_prefix_workspace_bytes(int H, int C, int G, int Hkv, int D) {
  const int64_t rows = (int64_t)C * G;
  size_t n = 0;
  if (rows <= 192) {  // a window may bring it to the groups of eight
    const int groups = (int)((rows + 7) / 8), blocks = (H + C + 15) / 16;
    n = block_decode_cluster(D, groups, Hkv, blocks) ? 0 : block_decode_workspace_bytes(D, block_decode_grid(groups, Hkv, blocks));
    if (few_rows(H, C, G, Hkv, D, 0)) return n;
  }
  // without a window: the largest plan
  const size_t tiles = bp::plan_of(H, C, G, Hkv, D, 0, block_device_sms()).bytes;
  return n > tiles ? n : tiles;
}

cudaError_t launch_block_prefix(BlockDecodeParams p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.C * p.G;
  if (few_rows(p.H, p.C, p.G, p.Hkv, p.D, p.window)) {
    p.B = (int)((rows + 7) / 8);
    p.HG = 1;
    p.HH = p.Hkv;
    p.max_blocks = (p.H + p.C + 15) / 16;
    p.grid = block_decode_grid(p.B, p.HH, p.max_blocks);
    p.cluster = block_decode_cluster(p.D, p.B, p.HH, p.max_blocks);
    p.divGrid = FastDiv((uint32_t)(p.cluster ? p.HH : p.grid));
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
