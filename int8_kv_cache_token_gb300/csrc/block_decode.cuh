// block_decode.cuh -- decode attention over the block-scaled INT8 KV cache, with
// an optional tanh cap, distance bias, sliding window and first visible key (the
// kernels; block_decode.cu instantiates them for 8 query rows per pass,
// block_decode_wide.cu for 16).
//
// For sequence b (position L - 1) and query head h, over the visible keys
// max(begin_b, L - window, 0) <= t < L:
//   s_t = cap tanh(x_t / cap) (or x_t),  x_t = scale q . (sK cK_t)
//   s_t -= slope_h (L - 1 - t);   O = sum_t softmax(s)_t sV cV_t
// with cK, cV the int8 codes and sK, sV the scales of the 16-token block of t.
//
// One 16-token block is one K = 16 step of an f16 MMA, so its two scales are
// one number each for the whole step: sK multiplies the finished scores, and
// sV joins the exponent.  With u_t = s_t log2 e + log2 sV the weights are
//   w_t = 2^(u_t - M),   O = sum w_t cV_t / sum w_t / sV
// for a running maximum M of u: the weights that meet the codes are at most
// one (times 2^8, below) whatever the scales are.  The codes are exact in f16,
// and so is q after a power-of-two scaling of its row; w is rounded to f16
// (2^-12 relative; for an fp32 output it is split into two f16 parts, 2^-22).
// M moves only when some u passes it by more than 8, so the output is rarely
// rescaled and the common step has no reduction across lanes at all.
//
// Every warp is a flash-decoding stream of its own: it takes every kWarps-th
// block of its CTA's range, has its own ring of page slots filled by its own
// bulk copies (lane 0), its own M, l and o in registers, and meets the other
// warps only at the end of a (sequence, KV head) pair.  The flattened list of
// all visible blocks of all pairs is cut evenly over the CTAs (one per SM), so
// ragged batches and single long sequences fill the GPU alike; a pair that
// spans CTAs leaves (o, M, l) records that a second kernel merges in CTA
// order.  Calls that few SMs finish sooner take a cluster per pair instead, joined
// through distributed shared memory in the same launch.
//
// Bound by HBM: 16 sequences of 32768 tokens (32/8/128) 164 us, 6.6 TB/s, 0.97 of
// the measured copy rate; 64 ragged ones (24/4/256, slopes) 330 us, 0.99 (the page
// copies' evict-first policy is worth 2 %).  One
// sequence of 4096 (24/4/256) 10 us, all of it latency: lengths, table, pages, a
// block's scores and products (0.8 us), the join.  A block of 16 tokens costs a
// warp about 450 instructions at head_dim 256, a third of the issue slots at the
// full HBM rate, so the conversions to f16 stay behind the copies.
//
// More than eight query heads of a KV head (or rows of a chunk) come as sixteen per
// pass where the blocks are many: the page is read and converted once for two tiles of
// the MMA, whose q then comes from shared memory, as o takes the registers.  750
// instructions a block at head_dim 256; what bounds it is their latency, two warps
// per scheduler issuing in 44 % of the cycles (16 sequences of 32768 tokens, 24/2/256:
// 99 us, 5.4 TB/s; 174 with eight rows per pass).
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace i8kv {
namespace {

constexpr int kBS = 16;
constexpr float kLazy = 8.0f;    // log2 units by which a score may pass M
constexpr int kMaxCluster = 8;
constexpr int kRounds = 6;       // most blocks per warp with a cluster per pair

// R: query rows per pass, 8 or 16 (one or two tiles of the MMA's N = 8).
template <int D, int R>
struct Geo {
  static constexpr int kTiles = R / 8;
  static constexpr int kWarps = D == 256 ? 8 : D * kTiles == 256 ? 12 : 16;  // by the registers that o takes
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kPage = D * kBS;
  static constexpr int kStages = 6144 / (D * kWarps);  // pages in flight per warp: 96 KB of each kind
  static constexpr int kStage = 2 * kPage;
  static constexpr int kRow = D + 4;                  // floats per head of a merge buffer (conflict-free)
  static constexpr int kBufs = D * kTiles > 128 && R > 8 ? 2 : 4;  // merge buffers
  static constexpr int oRing = 0;
  static constexpr int oMerge = oRing + kWarps * kStages * kStage;  // between joins: q of 16 rows
  static constexpr int oScale = oMerge + kBufs * R * kRow * 4;      // float2 (sK, sV) per stage
  static constexpr int oBar = oScale + kWarps * kStages * 8;
  static constexpr int oStat = oBar + kWarps * kStages * 8;         // M, l [kWarps][R] each
  static constexpr int oScan = oStat + 2 * (kWarps + 1) * R * 4;
  static constexpr int oQs = oScan + 64 * 4;                        // [16]: the factors of 16 rows' scores
  static constexpr int kTotal = oQs + (R > 8 ? R * 4 : 0);
  static_assert(kTotal <= 232448, "shared memory");
};

// The workspace: where every CTA's range starts (cuts [grid + 1] and a header
// each), then two partial records per CTA (its first and its last segment), each
// o [R][D], M [R], l [R].
struct Head {
  int b, hh;   // entry and head pass in which the range starts
  int first;   // visible blocks of the pair before the range
  int nb;      // visible blocks of the pair
};
static_assert(sizeof(Head) == 16, "16-byte aligned records");
__host__ __device__ constexpr int rec_floats(int D, int R) { return R * D + 2 * R; }
__host__ __device__ constexpr size_t cuts_bytes(int grid) { return (size_t)(grid + 4) / 4 * 16; }
__device__ __forceinline__ int* cuts_of(const BlockDecodeParams& p) { return static_cast<int*>(p.ws); }
__device__ __forceinline__ Head* heads_of(const BlockDecodeParams& p) {
  return reinterpret_cast<Head*>(static_cast<uint8_t*>(p.ws) + cuts_bytes(p.grid));
}
__device__ __forceinline__ float* record(const BlockDecodeParams& p, int slot, int D, int R) {
  return reinterpret_cast<float*>(heads_of(p) + p.grid) + (size_t)slot * rec_floats(D, R);
}

// One entry of the work list: a sequence (decode), or R (token, head) rows of
// a chunk, which then share a table and a head pass per KV head.
struct Seq {
  int lo, hi;        // keys [lo, hi) are visible to some row
  int lo_in, hi_in;  // keys [lo_in, hi_in) are visible to every row
  int fb, nb;        // blocks [fb, fb + nb) hold [lo, hi)
};

// Keys [lo, hi) that chunk row j (position H + j) sees.
__device__ __forceinline__ void chunk_interval(const BlockDecodeParams& p, int j, int& lo, int& hi) {
  lo = 0;
  if (p.window > 0) lo = max(0, p.H + j - p.window + 1);
  if (p.key_begin != nullptr) lo = max(lo, p.key_begin[j]);
  hi = p.H + j + 1;
  if (p.key_end != nullptr) hi = max(0, min(p.key_end[j], p.H + p.C));
}

template <bool kChunk, int R>
__device__ __forceinline__ Seq seq_of(const BlockDecodeParams& p, int b) {
  Seq s;
  if constexpr (kChunk) {
    s.lo = s.hi_in = 0x7fffffff;
    s.hi = s.lo_in = 0;
    const int j1 = min(p.C - 1, (b * R + R - 1) / p.G);
    for (int j = b * R / p.G; j <= j1; ++j) {
      int lo, hi;
      chunk_interval(p, j, lo, hi);
      s.lo_in = max(s.lo_in, lo);
      s.hi_in = min(s.hi_in, hi);
      if (lo < hi) {
        s.lo = min(s.lo, lo);
        s.hi = max(s.hi, hi);
      }
    }
  } else {
    s.hi = s.hi_in = max(0, min(p.seq_lens[b], p.max_blocks * kBS));
    s.lo = 0;
    if (p.window > 0) s.lo = max(0, s.hi - p.window);
    if (p.key_begin != nullptr) s.lo = max(s.lo, p.key_begin[b]);
    s.lo_in = s.lo;
  }
  if (s.lo >= s.hi) {
    s.fb = s.nb = 0;
  } else {
    s.fb = s.lo / kBS;
    s.nb = (s.hi + kBS - 1) / kBS - s.fb;
  }
  return s;
}

// Row c (0 .. R - 1) of head pass hh of entry b: its token (the row of q and out
// and of the masks) and query head; false where there is none.
template <bool kChunk, int R>
__device__ __forceinline__ bool row_of(const BlockDecodeParams& p, int b, int hh, int c, int& tok, int& head) {
  if constexpr (kChunk) {
    const int r = b * R + c;
    tok = p.divG.div(r);
    head = hh * p.G + r - tok * p.G;
    return r < p.C * p.G;
  } else {
    const int kvh = p.divHG.div(hh), in = (hh - kvh * p.HG) * R + c;
    tok = b;
    head = kvh * p.G + in;
    return in < p.G;
  }
}

// A warp's walk over the blocks of its CTA's range [u, u1) of the flattened
// list (sequence, head pass, block).
struct Walk {
  int b, hh;          // current sequence and head pass
  int left;           // blocks of the range from here on, this segment's included
  Seq s;
  int first, len;     // this segment: visible blocks [first, first + len) of the sequence
};

__device__ __forceinline__ void walk_segment(Walk& w) {
  w.len = min(w.s.nb - w.first, w.left);
}
// To the next segment; false at the end of the range.
template <bool kChunk, int R>
__device__ __forceinline__ bool walk_next(const BlockDecodeParams& p, Walk& w) {
  w.left -= w.len;
  if (w.left <= 0) return false;
  w.first = 0;
  if (++w.hh == p.HH) {
    w.hh = 0;
    do {
      if (++w.b >= p.B) return false;  // only if the lengths changed under the kernel
      w.s = seq_of<kChunk, R>(p, w.b);
    } while (w.s.nb == 0);
  }
  walk_segment(w);
  return true;
}

// The cut of `total` blocks over `grid` CTAs: the first total % grid take one more.
struct Cuts {
  int per, rem;
  __device__ __forceinline__ int at(int c) const { return per * c + min(c, rem); }
};
__device__ __forceinline__ Cuts cuts_for(const BlockDecodeParams& p, int total) {
  const int per = p.divGrid.div(total);
  return Cuts{per, total - per * p.grid};
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Sum over the CTA's threads, and the sum over the threads before this one.
template <int NW>
__device__ __forceinline__ int cta_scan(int v, int& before, int* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = warp_scan(v);
  __syncthreads();
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < warp) base += buf[i];
    total += buf[i];
  }
  before = base + x - v;
  return total;
}

// A place in the list: block `first` of a pair's nb.
struct Place {
  int u, b, hh, first, nb;
};
// A cut near the border between two pairs moves there, by up to kSnap blocks and
// half a range: the CTA would else have a segment more, whose join of the warps
// and record cost about as much as one more round of blocks over the warps (2 us).
template <int kSnap>
__device__ __forceinline__ void snap(Place& at, int per) {
  const int reach = min(kSnap, (per + 1) / 2);
  if (at.first <= reach && at.first < at.nb) {
    at.u -= at.first;
    at.first = 0;
  } else if (at.nb - at.first <= reach) {
    at.u += at.nb - at.first;
    at.first = at.nb;
  }
}
// The CTA's range: from `from` to block `to` of the list; whether some entry has
// no visible key.
struct Start {
  Place from;
  int to;
  bool empty;
};
// Up to kFew entries: each warp by itself, in one round of loads (no barrier).
// More: the CTA's threads together.
constexpr int kFew = 128;
template <bool kChunk, int R, int NW>
__device__ __forceinline__ Start find_start(const BlockDecodeParams& p, int* buf) {
  Start r{};
  Place at[2];
  const int tid = threadIdx.x, lane = tid & 31, c = blockIdx.x;
  int total = 0;
  Cuts cuts;
  if (p.B <= kFew) {
    int nb[kFew / 32], upto[kFew / 32];
#pragma unroll
    for (int k = 0; k < kFew / 32; ++k) nb[k] = 32 * k + lane < p.B ? seq_of<kChunk, R>(p, 32 * k + lane).nb : -1;
#pragma unroll
    for (int k = 0; k < kFew / 32; ++k) {
      if (32 * k >= p.B) continue;
      r.empty |= __any_sync(0xffffffffu, nb[k] == 0);
      upto[k] = total + warp_scan(max(nb[k], 0));
      total = __shfl_sync(0xffffffffu, upto[k], 31);
    }
    total *= p.HH;
    cuts = cuts_for(p, total);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      at[e] = Place{cuts.at(c + e), 0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kFew / 32; ++k) {
        if (32 * k >= p.B) continue;
        const int s0 = (upto[k] - max(nb[k], 0)) * p.HH;
        const uint32_t who = __ballot_sync(0xffffffffu, nb[k] > 0 && at[e].u >= s0 && at[e].u < upto[k] * p.HH);
        if (who) {
          const int l = __ffs(who) - 1, in = at[e].u - __shfl_sync(0xffffffffu, s0, l);
          at[e].nb = __shfl_sync(0xffffffffu, nb[k], l);
          at[e].b = 32 * k + l;
          at[e].hh = in / at[e].nb;
          at[e].first = in - at[e].hh * at[e].nb;
        }
      }
    }
  } else {
    int before;
    for (int b0 = 0; b0 < p.B; b0 += NW * 32)
      total += cta_scan<NW>(b0 + tid < p.B ? seq_of<kChunk, R>(p, b0 + tid).nb : 0, before, buf);
    total *= p.HH;
    cuts = cuts_for(p, total);
    r.empty = true;
    Place* found = reinterpret_cast<Place*>(buf + 32);
    if (tid < 2) found[tid] = Place{cuts.at(c + tid), 0, 0, 0, 0};
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += NW * 32) {
      const int nb = b0 + tid < p.B ? seq_of<kChunk, R>(p, b0 + tid).nb : 0;
      const int here = cta_scan<NW>(nb, before, buf);
      const int s0 = (run + before) * p.HH;
      for (int e = 0; e < 2; ++e) {
        const int u = cuts.at(c + e);
        if (u >= s0 && u < s0 + nb * p.HH) found[e] = Place{u, b0 + tid, (u - s0) / nb, (u - s0) % nb, nb};
      }
      run += here;
    }
    __syncthreads();
    at[0] = found[0];
    at[1] = found[1];
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (at[e].u > 0 && at[e].u < total) snap<NW>(at[e], cuts.per);
  r.from = at[0];
  r.to = at[1].u;
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The part of p that f16 leaves over, as f16x2 (hi is the packed f16 of (a, b)).
__device__ __forceinline__ uint32_t f16x2_rest(uint32_t hi, float a, float b) {
  float fa, fb;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(fa), "=f"(fb) : "r"(hi));
  return f16x2_of(a - fa, b - fb);
}

// kCap: scores pass through cap tanh(. / cap).  kHiLo: w as two f16 parts.
// Shared memory of the cluster's CTA `rank`, and its barrier.
__device__ __forceinline__ float4 peer_float4(const void* mine, int rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(smem_u32(mine)), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ float peer_float(const void* mine, int rank) {
  float v;
  asm volatile("{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v)
               : "r"(smem_u32(mine)), "r"(rank)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// kChunk: the work list holds the rows of one sequence's chunk.
// kCluster: a cluster of p.cluster CTAs per pair instead of the evenly cut list.
// The pair's blocks are shared out over the cluster, which joins its results
// through distributed shared memory: no records, no second kernel, no look at the
// other sequences' lengths.
template <int D, int R, bool kChunk, bool kCap, bool kHiLo, bool kCluster>
__global__ void __launch_bounds__(Geo<D, R>::kThreads, 1) block_decode_kernel(BlockDecodeParams p) {
  using Gm = Geo<D, R>;
  constexpr int NW = Gm::kWarps, NS = Gm::kStages, NT = Gm::kTiles;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + Gm::oRing + (size_t)warp * NS * Gm::kStage;
  float* merge = reinterpret_cast<float*>(smem + Gm::oMerge);
  float2* scl = reinterpret_cast<float2*>(smem + Gm::oScale) + warp * NS;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Gm::oBar) + warp * NS;
  float* statM = reinterpret_cast<float*>(smem + Gm::oStat);
  float* statL = statM + NW * R;
  float* joint = statL + NW * R;  // M, l of the segment
  int* scan = reinterpret_cast<int*>(smem + Gm::oScan);

  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  Walk w;
  const int cl_rank = kCluster ? (int)(blockIdx.x & (p.cluster - 1)) : 0;
  if constexpr (kCluster) {
    const int pair = blockIdx.x / p.cluster;  // a power of two
    w.b = p.divGrid.div(pair);                // by HH
    w.hh = pair - w.b * p.HH;
    w.s = seq_of<kChunk, R>(p, w.b);
    if (!kChunk && tid == 0 && cl_rank == 0 && w.hh == 0 && p.seq_lens[w.b] > p.max_blocks * kBS) record_error(2);
    if (w.s.nb == 0) {  // the whole cluster leaves
      if (cl_rank == 0)
        for (int i = tid; i < R * (D / 4); i += Gm::kThreads) {
          int tok, hd;
          if (row_of<kChunk, R>(p, w.b, w.hh, i / (D / 4), tok, hd))
            store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + (i % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
        }
      return;
    }
    w.first = w.s.nb * cl_rank / p.cluster;
    w.left = w.len = w.s.nb * (cl_rank + 1) / p.cluster - w.first;
  } else {
  // ---- this CTA's range of the flattened list, and where it starts ----
  const Start at = find_start<kChunk, R, NW>(p, scan);
  if (!kChunk && blockIdx.x == 0)
    for (int b = tid; b < p.B; b += Gm::kThreads)
      if (p.seq_lens[b] > p.max_blocks * kBS) record_error(2);
  if (at.empty)  // entries without a visible key: zero rows
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
      if (seq_of<kChunk, R>(p, b).nb == 0)
        for (int i = tid; i < p.HH * R * (D / 4); i += Gm::kThreads) {
          const int c4 = (i % (D / 4)) * 4, c = i / (D / 4);
          int tok, hd;
          if (row_of<kChunk, R>(p, b, c / R, c % R, tok, hd))
            store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + c4, make_float4(0.f, 0.f, 0.f, 0.f));
        }
  if (tid == 0) cuts_of(p)[blockIdx.x] = at.from.u;
  if (tid == 0 && blockIdx.x + 1 == gridDim.x) cuts_of(p)[gridDim.x] = at.to;
  if (at.from.u >= at.to) return;
  w.b = at.from.b;
  w.hh = at.from.hh;
  w.first = at.from.first;
  w.left = at.to - at.from.u;
  w.len = 0;
  w.s = seq_of<kChunk, R>(p, w.b);
  walk_segment(w);
  if (w.len == 0 && !walk_next<kChunk, R>(p, w)) return;  // the range starts with the next pair
  if (tid == 0) heads_of(p)[blockIdx.x] = Head{w.b, w.hh, w.first, w.s.nb};
  }

  // The query rows of a segment as they are.  Eight rows: every warp has them all
  // for itself, row g, dims 16 i + 4 t4 .. + 3.  Sixteen: a warp has rows warp + NW k,
  // four dims 4 (lane + 32 j) .. + 3 per lane, for the CTA's copy in shared memory.
  constexpr bool kShareQ = NT > 1;
  constexpr int kMine = (R + NW - 1) / NW, kPart = (D + 127) / 128;
  uint2 raw[kShareQ ? kMine * kPart : D / 16];
  auto load_q = [&](const Walk& x) {
    int tok, hd;
    if constexpr (kShareQ) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const bool in = row_of<kChunk, R>(p, x.b, x.hh, warp + NW * k, tok, hd) && warp + NW * k < R;
        const uint2* src = reinterpret_cast<const uint2*>(p.q + (int64_t)tok * p.q_stride + (size_t)hd * D);
#pragma unroll
        for (int j = 0; j < kPart; ++j) {
          raw[k * kPart + j] = make_uint2(0, 0);
          if (in && lane + 32 * j < D / 4) raw[k * kPart + j] = __ldg(src + lane + 32 * j);
        }
      }
    } else {
      const bool in = row_of<kChunk, R>(p, x.b, x.hh, g, tok, hd);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        raw[i] = make_uint2(0, 0);
        if (in) raw[i] = __ldg(reinterpret_cast<const uint2*>(p.q + (int64_t)tok * p.q_stride + (size_t)hd * D + 16 * i + 4 * t4));
      }
    }
  };
  load_q(w);

  // ---- the page copies: a walk of their own, NS blocks ahead of the consumer ----
  const uint64_t once = policy_evict_first();  // a page is read once a call
  Walk c = w;
  int c_i = warp;        // next block of the segment for this warp
  int c_n = 0;           // blocks asked for so far (slot c_n % NS)
  bool c_more = true;    // false: the range is done, or a wait ran out of time
  int table = 0, table_at = -1;  // lane i: the table entry of the warp's block table_at + i of the segment
  auto issue = [&]() {
    if (!c_more) return;
    while (c_i >= c.len) {
      if (!walk_next<kChunk, R>(p, c)) {
        c_more = false;
        return;
      }
      c_i = warp;
      table_at = -1;
    }
    const int k = c_i / NW;
    if (table_at < 0 || k >= table_at + 32) {
      table_at = k;
      const int i = warp + (k + lane) * NW;
      table = 0;
      if (i < c.len) {
        table = p.block_tables[(kChunk ? 0 : (size_t)c.b * p.max_blocks) + c.s.fb + c.first + i];
        if (table < 0 || table >= p.num_blocks) {
          record_error(2);
          table = 0;  // some page of the pool: the result is undefined, the read is not
        }
      }
    }
    const int phys = __shfl_sync(0xffffffffu, table, k - table_at);
    const int kvh = kChunk ? c.hh : p.divHG.div(c.hh);
    const int slot = c_n % NS;
    const size_t ph = (size_t)phys * p.Hkv + kvh;
    if (lane == 0) mbar_expect_tx(&bar[slot], Gm::kStage);
    __syncwarp();
    if (lane == 0) {
      bulk_g2s_hint(ring + slot * Gm::kStage, p.k_cache + ph * Gm::kPage, Gm::kPage, &bar[slot], once);
      bulk_g2s_hint(ring + slot * Gm::kStage + Gm::kPage, p.v_cache + ph * Gm::kPage, Gm::kPage, &bar[slot], once);
    } else if (lane <= 2) {
      cp_async_4(lane == 1 ? &scl[slot].x : &scl[slot].y, (lane == 1 ? p.k_scale : p.v_scale) + ph, 4);
      cp_async_mbar_arrive(&bar[slot]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[slot]);
    c_i += NW;
    ++c_n;
  };
#pragma unroll 1
  for (int i = 0; i < NS; ++i) issue();

  // The tokens behind the rows of a score fragment: row g of the MMA's upper
  // half is token tok0, of the lower half tok1.  Each set of eight covers all
  // residues mod 8 (ldmatrix without bank conflicts), and rows 2t, 2t + 1 of a
  // half are neighbouring tokens of 4t .. 4t + 3, as the V fragments want them.
  const int pr = g >> 1;
  const int tok0 = 4 * pr + (g & 1) + (pr >= 2 ? 2 : 0);
  const int tok1 = 4 * pr + (g & 1) + (pr >= 2 ? 0 : 2);
  // lane -> row address of ldmatrix: matrices (upper, lower) x (chunk, chunk + 1)
  const int lm_row = lane & 7, lm_mat = lane >> 3, lp = lm_row >> 1;
  const int lm_tok = 4 * lp + (lm_row & 1) + (((lp >= 2) != ((lm_mat & 1) != 0)) ? 2 : 0);
  const uint32_t k_off = (uint32_t)((lm_mat >> 1) * (kBS * 16) + lm_tok * 16);
  const uint32_t v_off = (uint32_t)(lane * 16);  // four groups of eight dims

  int n = 0;  // blocks consumed
  bool dead = false;  // a wait ran out of time: no further wait or copy, the walk ends quickly
  bool first_seg = true;
  for (;;) {
    // ---- a segment: blocks [first, first + len) of sequence b for one head pass ----
    // rows 8 x + 2 t4 + e (x < NT, e < 2) are this lane's columns of the scores and
    // the output
    int lo_[NT][2], hi_[NT][2], pos[NT][2];
    float sl[NT][2], qs[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int tok, hd;
        lo_[x][e] = w.s.lo;
        hi_[x][e] = w.s.hi;
        pos[x][e] = w.s.hi - 1;
        sl[x][e] = 0.f;
        if (row_of<kChunk, R>(p, w.b, w.hh, 8 * x + 2 * t4 + e, tok, hd)) {
          if (p.slopes != nullptr) sl[x][e] = -__ldg(p.slopes + hd) * kLog2e;
          if constexpr (kChunk) {
            chunk_interval(p, tok, lo_[x][e], hi_[x][e]);
            pos[x][e] = p.H + tok;
          }
        }
      }
    // q as the B operand: dims 16 c + 4 t4 .. + 3 of chunk c for row g of a tile,
    // scaled by a power of two that brings the row's maximum near 2^14
    uint32_t qf[kShareQ ? 1 : D / 16][2];
    uint4* qsh = reinterpret_cast<uint4*>(merge);  // [chunk pair][tile][lane]
    auto peak = [](float am, uint2 r) {
      am = fmaxf(am, fmaxf(fabsf(__uint_as_float(r.x << 16)), fabsf(__uint_as_float(r.x & 0xffff0000u))));
      return fmaxf(am, fmaxf(fabsf(__uint_as_float(r.y << 16)), fabsf(__uint_as_float(r.y & 0xffff0000u))));
    };
    auto scaled = [](uint2 r, float up) {
      return make_uint2(f16x2_of(__uint_as_float(r.x << 16) * up, __uint_as_float(r.x & 0xffff0000u) * up),
                        f16x2_of(__uint_as_float(r.y << 16) * up, __uint_as_float(r.y & 0xffff0000u) * up));
    };
    auto factors = [&](float am, float& up) {  // up: the power of two; returns the scores' factor
      const int ex = max(-100, (int)(__float_as_uint(am) >> 23) - 127);  // -100: zero rows and values below 2^-100
      up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
      return __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * p.score_mul;
    };
    if constexpr (kShareQ) {
      float* qsc = reinterpret_cast<float*>(smem + Gm::oQs);
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int row = warp + NW * k;
        if (R % NW != 0 && row >= R) break;
        float am = 0.f, up;
#pragma unroll
        for (int j = 0; j < kPart; ++j) am = peak(am, raw[k * kPart + j]);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, d));
        const float f = factors(am, up);
        if (lane == 0) qsc[row] = f;
#pragma unroll
        for (int j = 0; j < kPart; ++j) {
          const int m = lane + 32 * j, ch = m >> 2;  // four dims of chunk ch for lane 4 (row % 8) + m % 4
          if (m < D / 4)
            reinterpret_cast<uint2*>(qsh)[(((ch >> 1) * NT + (row >> 3)) * 32 + (row & 7) * 4 + (m & 3)) * 2 + (ch & 1)] =
                scaled(raw[k * kPart + j], up);
        }
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) qs[x][e] = qsc[8 * x + 2 * t4 + e];
    } else {
      float am = 0.f, up;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) am = peak(am, raw[i]);
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const float f = factors(am, up);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint2 h = scaled(raw[i], up);
        qf[i][0] = h.x;
        qf[i][1] = h.y;
      }
      qs[0][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
      qs[0][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
    }
    float o[NT][D / 16][4], M[NT][2], l[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[x][i][j] = 0.f;
      M[x][0] = M[x][1] = -INFINITY;
      l[x][0] = l[x][1] = 0.f;
    }

    for (int i = warp; i < w.len; i += NW, ++n) {
      const int slot = n % NS;
      if (!dead && !mbar_wait(&bar[slot], (n / NS) & 1)) {
        dead = true;
        c_more = false;
      }
      const uint8_t* kp = ring + slot * Gm::kStage;
      const uint8_t* vp = kp + Gm::kPage;
      const float sk = scl[slot].x, sv = scl[slot].y;
      // scores: two chains over the even and odd chunks
      float s[NT][2][4];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[x][0][j] = s[x][1][j] = 0.f;
#pragma unroll
      for (int ch = 0; ch < D / 16; ch += 2) {
        uint32_t a[4], lo[4], hi[4];
        ldmatrix_x4(a, kp + ch * (kBS * 16) + k_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) s8x4_to_f16(a[j], lo[j], hi[j]);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          uint4 q;
          if constexpr (kShareQ)
            q = qsh[((ch >> 1) * NT + x) * 32 + lane];
          else
            q = make_uint4(qf[ch][0], qf[ch][1], qf[ch + 1][0], qf[ch + 1][1]);
          mma_f16_16816(s[x][0], lo[0], lo[1], hi[0], hi[1], q.x, q.y);
          mma_f16_16816(s[x][1], lo[2], lo[3], hi[2], hi[3], q.z, q.w);
        }
      }
      // u = score log2 e + log2 sV.  A block of zero V codes (sV = 0) gets the
      // floor 2^-100: its codes add nothing, its weights still count in l.
      const float svf = fmaxf(sv, kTinyDivisor);
      const float lv = kHiLo ? log2f(svf) : __log2f(svf), inv = __frcp_rn(svf);
      float u[NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) u[x][j] = (s[x][0][j] + s[x][1][j]) * (qs[x][j & 1] * sk);
      const int key0 = (w.s.fb + w.first + i) * kBS;
      if constexpr (kCap) {
        // u = score / cap here; cap log2 e tanh u, by the polynomial in u^2 for |u| <= 1
        bool in = true;
#pragma unroll
        for (int x = 0; x < NT; ++x)
          in = in && fmaxf(fmaxf(fabsf(u[x][0]), fabsf(u[x][1])), fmaxf(fabsf(u[x][2]), fabsf(u[x][3]))) <= 1.f;
        if (__any_sync(0xffffffffu, !in)) {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              u[x][j] = kHiLo ? __fmaf_rn(p.cap_log2, tanhf(u[x][j]), lv)
                              : __fmaf_rn(-2.f * p.cap_log2, rcp_approx(ex2(u[x][j] * (2.f * kLog2e)) + 1.f), p.cap_log2 + lv);
        } else {
#pragma unroll
          for (int x = 0; x < NT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float y = u[x][j] * u[x][j];
              float a = p.cap_poly[kCapDeg];
#pragma unroll
              for (int d = kCapDeg - 1; d >= 0; --d) a = __fmaf_rn(a, y, p.cap_poly[d]);
              u[x][j] = __fmaf_rn(a, u[x][j], lv);
            }
        }
      } else {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) u[x][j] += lv;
      }
      // u[x][j] belongs to key key0 + (j < 2 ? tok0 : tok1) and row 8 x + 2 t4 + j % 2
      if (p.slopes != nullptr) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[x][j] = __fmaf_rn(sl[x][j & 1], (float)abs(key0 + (j < 2 ? tok0 : tok1) - pos[x][j & 1]), u[x][j]);
      }
      if (key0 < w.s.lo_in || key0 + kBS > w.s.hi_in) {  // a block with hidden tokens
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = key0 + (j < 2 ? tok0 : tok1);
            if (key < lo_[x][j & 1] || key >= hi_[x][j & 1]) u[x][j] = -INFINITY;
          }
      }
      // M moves for all the lanes of a head together
      bool over = false;
#pragma unroll
      for (int x = 0; x < NT; ++x)
        over = over || fmaxf(u[x][0], u[x][2]) > M[x][0] + kLazy || fmaxf(u[x][1], u[x][3]) > M[x][1] + kLazy;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          float m[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) m[e] = fmaxf(M[x][e], fmaxf(u[x][e], u[x][e + 2]));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
            m[1] = fmaxf(m[1], __shfl_xor_sync(0xffffffffu, m[1], d));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = M[x][e] == -INFINITY ? 0.f : ex2(M[x][e] - m[e]);
            M[x][e] = m[e];
            l[x][e] *= a;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              o[x][k][e] *= a;
              o[x][k][e + 2] *= a;
            }
          }
        }
      }
      uint32_t bw[NT][2], rest[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        // a row that has seen no key yet: M = -inf, weights 0
        const float n0 = kChunk && M[x][0] == -INFINITY ? 0.f : M[x][0], n1 = kChunk && M[x][1] == -INFINITY ? 0.f : M[x][1];
        const float w0 = ex2(u[x][0] - n0), w1 = ex2(u[x][1] - n1), w2 = ex2(u[x][2] - n0), w3 = ex2(u[x][3] - n1);
        l[x][0] = __fmaf_rn(w0 + w2, inv, l[x][0]);
        l[x][1] = __fmaf_rn(w1 + w3, inv, l[x][1]);
        // [token][head] -> the B operand [head][token pairs]; for t4 >= 2 the upper
        // half holds tokens 4 t4 + 2, + 3
        const uint32_t p0 = f16x2_of(w0, w1), p1 = f16x2_of(w2, w3);
        const uint32_t x0 = movmatrix_trans(p0), x1 = movmatrix_trans(p1);
        bw[x][0] = t4 < 2 ? x0 : x1;
        bw[x][1] = t4 < 2 ? x1 : x0;
        if constexpr (kHiLo) {
          const uint32_t y0 = movmatrix_trans(f16x2_rest(p0, w0, w1)), y1 = movmatrix_trans(f16x2_rest(p1, w2, w3));
          rest[x][0] = t4 < 2 ? y0 : y1;
          rest[x][1] = t4 < 2 ? y1 : y0;
        }
      }
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) {  // 32 dims: two row tiles of the MMA
        uint32_t a[4], lo[4], hi[4];
        ldmatrix_x4(a, vp + dt * (32 * 16) + v_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) s8x4_to_f16(a[j], lo[j], hi[j]);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          mma_f16_16816(o[x][2 * dt], lo[0], lo[1], hi[0], hi[1], bw[x][0], bw[x][1]);
          mma_f16_16816(o[x][2 * dt + 1], lo[2], lo[3], hi[2], hi[3], bw[x][0], bw[x][1]);
        }
        if constexpr (kHiLo) {
#pragma unroll
          for (int x = 0; x < NT; ++x) {
            mma_f16_16816(o[x][2 * dt], lo[0], lo[1], hi[0], hi[1], rest[x][0], rest[x][1]);
            mma_f16_16816(o[x][2 * dt + 1], lo[2], lo[3], hi[2], hi[3], rest[x][0], rest[x][1]);
          }
        }
      }
      __syncwarp();  // every lane is done with the slot
      issue();
    }

    // the next segment's query rows arrive during the join (sixteen of them; eight take
    // the registers of the join: 170 against 165 us for 16 sequences of 32768, 32/8/128)
    Walk nx = w;
    bool more = false;
    if constexpr (!kCluster && kShareQ) {
      more = walk_next<kChunk, R>(p, nx);
      if (more) load_q(nx);
    }
    // ---- the warps' (o, M, l) of this segment joined, in a fixed order ----
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], d);
        if (g == 0) {
          statM[warp * R + 8 * x + 2 * t4 + e] = M[x][e];
          statL[warp * R + 8 * x + 2 * t4 + e] = l[x][e];
        }
      }
    __syncthreads();
    float f[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float C = -INFINITY;
#pragma unroll
        for (int i = 0; i < NW; ++i) C = fmaxf(C, statM[i * R + 8 * x + 2 * t4 + e]);
        f[x][e] = M[x][e] == -INFINITY ? 0.f : ex2(M[x][e] - C);
      }
    // Each head's maximum and sum, once, by R lanes of the last warp.
    if (warp == NW - 1 && lane < R) {
      float C = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) C = fmaxf(C, statM[k * R + lane]);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float m = statM[k * R + lane];
        if (m != -INFINITY) sum = __fmaf_rn(statL[k * R + lane], ex2(m - C), sum);
      }
      joint[lane] = C;
      joint[R + lane] = sum;
    }
    // The CTA's last segment has the page ring to itself: a buffer per warp, one
    // round.  Before that the next segment's pages are on their way into the ring,
    // and kBufs warps at a time add to as many buffers.
    const bool end = w.left == w.len;
    const int bufs = end ? NW : Gm::kBufs, rounds = NW / bufs;
    float* joined = end ? reinterpret_cast<float*>(smem + Gm::oRing) : merge;
    float* buf = joined + (warp % bufs) * (R * Gm::kRow);
#pragma unroll 1
    for (int r = rounds - 1; r >= 0; --r) {  // the last warps first
      if (warp / bufs == r) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float& x = buf[(8 * t + 2 * t4 + (j & 1)) * Gm::kRow + 16 * k + g + (j >> 1) * 8];
              x = __fmaf_rn(o[t][k][j], f[t][j & 1], r == rounds - 1 ? 0.f : x);
            }
      }
      __syncthreads();
    }
    if constexpr (kCluster) {
      // this CTA's sum in the first buffer, then every CTA joins a share of the columns
      for (int i = tid; i < R * D / 4; i += Gm::kThreads) {
        float4* x = reinterpret_cast<float4*>(joined + i / (D / 4) * Gm::kRow + (i % (D / 4)) * 4);
        float4 acc = *x;
#pragma unroll 4
        for (int k = 1; k < bufs; ++k) {
          const float4 y = x[k * (R * Gm::kRow / 4)];
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
        }
        *x = acc;
      }
      cluster_sync();
      for (int i = cl_rank * Gm::kThreads + tid; i < R * D / 4; i += p.cluster * Gm::kThreads) {
        const int h = i / (D / 4), c4 = (i % (D / 4)) * 4;
        int tok, hd;
        if (!row_of<kChunk, R>(p, w.b, w.hh, h, tok, hd)) continue;
        float m[kMaxCluster], l = 0.f, C = -INFINITY;
        float4 x[kMaxCluster], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < p.cluster) {
            m[k] = peer_float(joint + h, k);
            x[k] = peer_float4(joined + h * Gm::kRow + c4, k);
            C = fmaxf(C, m[k]);
          }
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k)
          if (k < p.cluster && m[k] != -INFINITY) {
            const float f = ex2(m[k] - C);
            l = __fmaf_rn(peer_float(joint + R + h, k), f, l);
            acc.x = __fmaf_rn(x[k].x, f, acc.x);
            acc.y = __fmaf_rn(x[k].y, f, acc.y);
            acc.z = __fmaf_rn(x[k].z, f, acc.z);
            acc.w = __fmaf_rn(x[k].w, f, acc.w);
          }
        const float iv = l > 0.f ? 1.0f / l : 0.f;  // a row without a visible key is zero
        store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + c4,
                   make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv));
      }
      cluster_sync();  // the peers have read this CTA's results
      break;
    }
    const bool whole = w.first == 0 && w.len == w.s.nb;
    float* rec = record(p, 2 * blockIdx.x + (first_seg ? 0 : 1), D, R);
    for (int i = tid; i < R * D / 4; i += Gm::kThreads) {
      const int h = i / (D / 4), c4 = (i % (D / 4)) * 4;
      int tok, hd;
      if (!row_of<kChunk, R>(p, w.b, w.hh, h, tok, hd)) continue;
      float4 acc = *reinterpret_cast<const float4*>(joined + h * Gm::kRow + c4);
#pragma unroll 4
      for (int k = 1; k < bufs; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(joined + (k * R + h) * Gm::kRow + c4);
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      const float C = joint[h], l = joint[R + h];
      if (whole) {
        const float iv = l > 0.f ? 1.0f / l : 0.f;  // a row without a visible key is zero
        store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + c4,
                   make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv));
      } else {
        *reinterpret_cast<float4*>(rec + h * D + c4) = acc;
        if (c4 == 0) {
          rec[R * D + h] = C;
          rec[R * D + R + h] = l;
        }
      }
    }
    first_seg = false;
    if constexpr (kShareQ) {
      if (!more) break;
      w = nx;
    } else {
      if (!walk_next<kChunk, R>(p, w)) break;
      load_q(w);
    }
    __syncthreads();  // the merge buffers are free again
  }
  // after a time-out: the copies still under way get one more (bounded) wait
  if (__any_sync(0xffffffffu, dead))
    for (int k = max(0, c_n - NS); k < c_n; ++k) mbar_wait(&bar[k % NS], (k / NS) & 1);
}

// The records of the pairs that span CTAs, merged in CTA order.  A pair is cut
// only where a CTA's range starts, so the grid runs over those places and rows;
// the first cut inside a pair has its merge.  kParts threads per four columns, each
// with every kParts-th record, six in flight; a CTA has kMergeThreads / kParts rows.
// From four pairs on, kParts = 4: a pair then has 38 records or fewer on average, and
// the CTAs of many rows come in half as many waves (24 pairs of 16 rows at head_dim
// 256 41.8 -> 39.0 us); below, 8 (2 pairs 19.0 us against 21.1).
constexpr int kMergeThreads = 8;  // per four columns

template <int D, int R, bool kChunk, int kParts>
__global__ void __launch_bounds__(D / 4 * kMergeThreads) block_decode_merge_kernel(BlockDecodeParams p, int rows) {
  constexpr int kCols = D / 4, kThreads = kCols * kMergeThreads, kRows = kMergeThreads / kParts;
  __shared__ float4 s_o[kRows][kParts][kCols];
  __shared__ float s_ml[kRows][kParts][2];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, grid = p.grid;
  const int sets = (rows + kRows - 1) / kRows, cut = blockIdx.x / sets + 1;
  const int col = tid % kCols, part = tid / kCols % kParts, mine = tid / (kCols * kParts);
  const int h = (blockIdx.x - (cut - 1) * sets) * kRows + mine;
  const int* cuts = cuts_of(p);
  const int here = cuts[cut], prev = cuts[cut - 1], next = cuts[cut + 1];
  const Head hd = heads_of(p)[cut];
  const int later = cut + 1 + tid < grid ? cuts[cut + 1 + tid] : 0x7fffffff;
  if (here >= next || hd.first == 0) return;  // an empty range, or no pair is cut here
  const int a = here - hd.first, e = a + hd.nb;  // the pair's blocks of the list
  if (prev > a) return;  // not the first cut of the pair
  int tok, qh;
  const bool in = h < rows && row_of<kChunk, R>(p, hd.b, hd.hh, h, tok, qh);
  // CTA c0 has the pair's beginning (cuts inside a pair differ, so it is the one
  // before); c1 is the last whose range starts before the pair's end
  const int c0 = cut - 1;
  int c1 = cut + __syncthreads_count(later < e);
  for (int c = cut + 1 + kThreads; c < grid; c += kThreads) c1 += __syncthreads_count(c + tid < grid && cuts[c + tid] < e);
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = in ? c0 + part : c1 + 1; c <= c1; c += 6 * kParts) {
    float4 x[6];
    float m[6], ll[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) {
      const int cc = c + k * kParts;
      m[k] = -INFINITY;
      if (cc <= c1) {
        // a CTA whose range starts inside the pair has it as its first segment
        const float* rec = record(p, 2 * cc + (cc > c0 || prev == a ? 0 : 1), D, R);
        x[k] = *reinterpret_cast<const float4*>(rec + h * D + 4 * col);
        m[k] = rec[R * D + h];
        ll[k] = rec[R * D + R + h];
      }
    }
#pragma unroll
    for (int k = 0; k < 6; ++k) {
      const float nm = fmaxf(M, m[k]);
      if (m[k] == -INFINITY) continue;
      const float f = ex2(M - nm), g = ex2(m[k] - nm);  // 2^-inf = 0
      acc.x = acc.x * f + x[k].x * g;
      acc.y = acc.y * f + x[k].y * g;
      acc.z = acc.z * f + x[k].z * g;
      acc.w = acc.w * f + x[k].w * g;
      l = l * f + ll[k] * g;
      M = nm;
    }
  }
  s_o[mine][part][col] = acc;
  if (col == 0) {
    s_ml[mine][part][0] = M;
    s_ml[mine][part][1] = l;
  }
  __syncthreads();
  if (part == 0 && in) {
    float C = -INFINITY;
#pragma unroll
    for (int k = 0; k < kParts; ++k) C = fmaxf(C, s_ml[mine][k][0]);
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      if (s_ml[mine][k][0] == -INFINITY) continue;
      const float f = ex2(s_ml[mine][k][0] - C);
      const float4 x = s_o[mine][k][col];
      r.x += x.x * f;
      r.y += x.y * f;
      r.z += x.z * f;
      r.w += x.w * f;
      den += s_ml[mine][k][1] * f;
    }
    const float iv = den > 0.f ? 1.0f / den : 0.f;
    store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + qh) * D + 4 * col, make_float4(r.x * iv, r.y * iv, r.z * iv, r.w * iv));
  }
}

template <int D, int R, bool kChunk, bool kCap, bool kHiLo, bool kCluster>
cudaError_t launch_c(const BlockDecodeParams& p, cudaStream_t stream) {
  auto* kernel = block_decode_kernel<D, R, kChunk, kCap, kHiLo, kCluster>;
  // the shared-memory opt-in, once per device (graph captures then make no attribute call)
  int dev = 0;
  cudaGetDevice(&dev);
  static bool opted[64] = {false};
  if (dev < 0 || dev >= 64 || !opted[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D, R>::kTotal);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) opted[dev] = true;
  }
  if constexpr (kCluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.B * p.HH * p.cluster);
    cfg.blockDim = dim3(Geo<D, R>::kThreads);
    cfg.dynamicSmemBytes = Geo<D, R>::kTotal;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  }
  const cudaError_t e = launch_pdl(kernel, dim3(p.grid), dim3(Geo<D, R>::kThreads), Geo<D, R>::kTotal, stream, p);
  if (e != cudaSuccess) return e;
  if (p.grid == 1) return cudaSuccess;
  const int rows = !kChunk && p.G < R ? p.G : R;
  const bool many = (long long)p.B * p.HH >= 4;
  return launch_pdl(many ? block_decode_merge_kernel<D, R, kChunk, 4> : block_decode_merge_kernel<D, R, kChunk, 8>,
                    dim3((p.grid - 1) * (many ? (rows + 1) / 2 : rows)), dim3(D / 4 * kMergeThreads), 0, stream, p, rows);
}

template <int D, int R, bool kChunk, bool kCap, bool kHiLo>
cudaError_t launch_d(const BlockDecodeParams& p, cudaStream_t stream) {
  return p.cluster ? launch_c<D, R, kChunk, kCap, kHiLo, true>(p, stream) : launch_c<D, R, kChunk, kCap, kHiLo, false>(p, stream);
}

template <int D, int R, bool kChunk>
cudaError_t launch_v(const BlockDecodeParams& p, cudaStream_t stream) {
  const bool cap = p.cap_log2 > 0.f;
  if (p.out_bf16) return cap ? launch_d<D, R, kChunk, true, false>(p, stream) : launch_d<D, R, kChunk, false, false>(p, stream);
  return cap ? launch_d<D, R, kChunk, true, true>(p, stream) : launch_d<D, R, kChunk, false, true>(p, stream);
}

template <int R>
cudaError_t launch_rows(const BlockDecodeParams& p, bool chunk, cudaStream_t stream) {
  if (p.D == 256) return chunk ? launch_v<256, R, true>(p, stream) : launch_v<256, R, false>(p, stream);
  if (p.D == 128) return chunk ? launch_v<128, R, true>(p, stream) : launch_v<128, R, false>(p, stream);
  return chunk ? launch_v<64, R, true>(p, stream) : launch_v<64, R, false>(p, stream);
}

}  // namespace
}  // namespace i8kv
