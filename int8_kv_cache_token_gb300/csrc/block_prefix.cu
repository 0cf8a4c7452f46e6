// block_prefix.cu -- the route of a chunk over the block-scaled cache, and its workspace.
#include "block_prefix.cuh"

namespace i8kv {

cudaError_t launch_block_prefix_64(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_128(const bp::Params& pp, cudaStream_t stream);
cudaError_t launch_block_prefix_256(const bp::Params& pp, cudaStream_t stream);

namespace {

// Few (token, head) rows of a KV head run in groups of 8 or 16, each reading the int8
// cache itself; more run in 128-row blocks on 16-bit operand tiles, which have to be
// made first.  Groups that have a cluster each take 8 to 20 us, less than the second
// way's three launches (24/4/256, 1000 keys, 192 rows 14 against 20 us).  On the evenly
// cut list, with X = keys x Hkv x D in millions and g groups of 16, they take about 20 +
// 0.36 g X us against 23 + 1.55 X (24/4/256, 8192 keys, 60 rows 28 against 36 us, 96
// rows 39 against 36.6; 32768 keys, 60 rows 66 against 77).  More (group, KV head) pairs
// than SMs pay for each pair's start and end (32/8/128, 384 rows without a history 34
// against 14 us), so beyond 64 rows the pairs have to fit.  The list of the groups'
// blocks is counted in 31 bits.
constexpr int kFewRows = 384;
bool few_rows(int H, int C, int G, int Hkv, int D, int window) {
  const int64_t rows = (int64_t)C * G, groups = (rows + 15) / 16;
  const int64_t keys = window > 0 && (int64_t)window < H ? (int64_t)window + C : (int64_t)H + C;
  if (2 * groups * Hkv * (((int64_t)H + C) / 16 + 1) >= (1ll << 31)) return false;
  if (groups <= 4) return true;
  if (rows > kFewRows) return false;
  const int blocks = (H + C + 15) / 16, R = block_decode_rows(D, (int)rows, 1, Hkv, blocks);
  if (block_decode_cluster(D, R, ((int)rows + R - 1) / R, Hkv, blocks)) return true;
  return groups * Hkv <= 128 && (4 * groups - 17) * keys * Hkv * D <= 33000000;
}

// CTAs for the row groups: they see about the same keys, so where an equal number of
// CTAs for each leaves few SMs over, no CTA has parts of two (and two joins).  That
// is worth 4 us, and the idle SMs cost less up to some sixteen rounds of blocks over a
// CTA's warps (16 pairs of 8192 keys, 32/8/128 24.0 -> 18.8 us; 32768 keys 43.2 -> 44.3).
int group_grid(int pairs, int blocks) {
  const int grid = block_decode_grid(pairs, 1, blocks), each = grid / pairs;
  return 16 * pairs * each >= 15 * grid && blocks <= 128 * each ? pairs * each : grid;
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
  if (rows <= kFewRows) {  // a window may bring it to the row groups
    const int blocks = (H + C + 15) / 16, R = block_decode_rows(D, (int)rows, 1, Hkv, blocks);
    const int groups = ((int)rows + R - 1) / R;
    n = block_decode_cluster(D, R, groups, Hkv, blocks) ? 0 : block_decode_workspace_bytes(D, R, group_grid(groups * Hkv, blocks));
    if (few_rows(H, C, G, Hkv, D, 0)) return n;
  }
  // without a window: the largest plan
  const size_t tiles = bp::plan_of(H, C, G, Hkv, D, 0, block_device_sms()).bytes;
  return n > tiles ? n : tiles;
}

cudaError_t launch_block_prefix(BlockDecodeParams p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.C * p.G;
  if (few_rows(p.H, p.C, p.G, p.Hkv, p.D, p.window)) {
    p.max_blocks = (p.H + p.C + 15) / 16;
    p.R = block_decode_rows(p.D, (int)rows, 1, p.Hkv, p.max_blocks);
    p.B = ((int)rows + p.R - 1) / p.R;
    p.HG = 1;
    p.HH = p.Hkv;
    p.grid = group_grid(p.B * p.HH, p.max_blocks);
    p.cluster = block_decode_cluster(p.D, p.R, p.B, p.HH, p.max_blocks);
    p.divGrid = FastDiv((uint32_t)(p.cluster ? p.HH : p.grid));
    return launch_block_rows(p, true, stream);
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
