// block_decode.cu -- the decode attention of block_decode.cuh with 8 query rows per
// pass, and its launch shapes.
#include "block_decode.cuh"

namespace i8kv {
I8KV_DEFINE_ERROR_ACCESSOR(read_error_block_decode)

// The SMs of the current device, asked once per device.
int block_device_sms() {
  static int known[64] = {0};
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && known[dev] > 0) return known[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 1;
  if (dev >= 0 && dev < 64) known[dev] = n;
  return n;
}

// CTAs of the attention kernel: one per SM, or one per block where there are fewer.
int block_decode_grid(int entries, int HH, int max_blocks) {
  const long long most = (long long)entries * HH * max_blocks;
  const int sms = block_device_sms();
  return most < sms ? (int)(most > 0 ? most : 1) : sms;
}

// How many clusters of c CTAs (one CTA per SM) run at once, asked once per device.
static int clusters_at_once(int c) {
  if (c == 1) return block_device_sms();
  static int known[64][kMaxCluster + 1] = {};
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 0;
  if (known[dev][c] > 0) return known[dev][c] - 1;
  auto* kernel = block_decode_kernel<256, 8, false, false, false, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCluster * 64);
  cfg.blockDim = dim3(Geo<256, 8>::kThreads);
  cfg.dynamicSmemBytes = Geo<256, 8>::kTotal;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<256, 8>::kTotal) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 0) {
    cudaGetLastError();
    return 0;
  }
  known[dev][c] = n + 1;
  return n;
}

// CTAs per pair with a cluster per pair (0: the evenly cut list): the most that
// run at once, if then no warp has more than kRounds blocks of the longest
// sequence that the table can hold (a round takes about 1 us, the list's second
// kernel and its look at all lengths about 3).  A call whose blocks the whole GPU
// needs is better cut evenly, whatever the lengths.  Measured: one sequence of 4096
// tokens (24/4/256) 10.1 us against 11.5 with the list, five of up to 777 (8/8/64)
// 6.8 against 8.7.
int block_decode_cluster(int D, int R, int entries, long long HH, int max_blocks) {
  const long long pairs = entries * HH;
  const int warps = R > 8 ? (D == 256 ? Geo<256, 16>::kWarps : D == 128 ? Geo<128, 16>::kWarps : Geo<64, 16>::kWarps)
                          : (D == 256 ? Geo<256, 8>::kWarps : D == 128 ? Geo<128, 8>::kWarps : Geo<64, 8>::kWarps);
  int c = kMaxCluster;
  while (c > 1 && pairs > clusters_at_once(c)) c >>= 1;
  if (pairs > clusters_at_once(c)) return 0;
  while (c > 1 && max_blocks <= (c / 2) * warps) c >>= 1;  // one round is enough
  return max_blocks <= kRounds * c * warps ? c : 0;
}

// Sixteen rows per pass read the pages of more than eight rows once, and cost 1.3 to
// 1.6 times the instructions per block, so they win where the blocks are many: from
// 32 of them per SM on (16 sequences of 32768 tokens, 64/4/128 164 -> 115 us, 24/2/256
// 174 -> 99 us; of 4096 tokens 30.7 -> 28.5 us; against that 16/1/128, 27 blocks per
// SM, 11.2 us with eight and 13.5 with sixteen), or where only the halved number of
// pairs has room for a cluster each (4 sequences of 4096 tokens, 24/2/256 18.7 -> 12.9 us).
int block_decode_rows(int D, int rows, int entries, int Hkv, int max_blocks) {
  if (rows <= 8) return 8;
  const long long narrow = (long long)Hkv * ((rows + 7) / 8), wide = (long long)Hkv * ((rows + 15) / 16);
  if ((long long)entries * wide * max_blocks >= 32ll * block_device_sms()) return 16;
  return !block_decode_cluster(D, 8, entries, narrow, max_blocks) && block_decode_cluster(D, 16, entries, wide, max_blocks) ? 16 : 8;
}

size_t block_decode_workspace_bytes(int D, int R, int grid) {
  return cuts_bytes(grid) + (size_t)grid * (sizeof(Head) + 2 * rec_floats(D, R) * sizeof(float));
}

cudaError_t launch_block_rows(const BlockDecodeParams& p, bool chunk, cudaStream_t stream) {
  return p.R > 8 ? launch_block_rows_wide(p, chunk, stream) : launch_rows<8>(p, chunk, stream);
}

}  // namespace i8kv
