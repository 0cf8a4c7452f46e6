// block_prefix.cuh -- chunk attention over the block-scaled INT8 KV cache on the
// 5th-generation tensor cores (the kernels; one .cu per head_dim instantiates them).
//
// Row (token j, query head h) at position pos = H + j over its visible keys:
//   x_t = scale q . (sK cK_t),  s_t = cap tanh(x_t / cap) (or x_t) - slope_h |pos - t|
//   O = sum_t softmax(s)_t sV cV_t
// as in block_decode.cuh: u_t = s_t log2 e + log2 sV, weights w_t = 2^(u_t - M),
// O = sum w cV / sum w / sV, so the two scales of a 16-key block are one multiply
// and one addend of its 16 scores, and the products below run on the bare codes.
//
// A CTA owns a row block, 128 (token, head) rows of one KV head (256 for head_dim
// up to 128), and walks 128-key tiles:
//   S = Q K^T    tcgen05, bf16 Q (as given) x bf16 codes (exact), M = N = 128, K = D
//   u, M, w      CUDA cores, one thread per row
//   O += W V     tcgen05, f16 W (from tensor memory) x f16 codes (exact), N = D
// S has two slots in tensor memory, so that one softmax runs beside the products
// of the other.  W overwrites its S slot.  With head_dim up to 128 the two are
// two 128-row halves of the row block, each with its warpgroup, S and O: every
// K / V tile that is loaded serves 256 rows.  A head_dim of 256 leaves room for one
// O: two warpgroups take alternate tiles of the same 128 rows and hand the running
// maximum on.  O is rescaled only when a row's maximum grows by more than 2^8.  For
// an fp32 output W is two f16 parts (2^-22 instead of 2^-12 relative), side by side
// in the slot.
//
// The codes become 16-bit operand tiles once per call (block_tiles_kernel), in
// the swizzled layout that the MMAs read, so a tile is one bulk copy per half and
// every row block of a KV head shares the conversion.
//
// All (KV head, row block, tile) steps form one list, cut evenly over one CTA per
// SM; row blocks that span CTAs leave (O, M, l) records, merged in CTA order by a
// third kernel.  So a causal triangle, a window, packed documents and a short
// chunk over a long history all fill the GPU.
//
// Warps: 0 tile copies, 1 MMA issue, 2 tensor memory, 4-7 and 8-11 softmax and
// query rows.  One thread issues both products: MMAs of a CTA execute in issue
// order, which is what lets W share its S slot with the S after next.
//
// What bounds it, measured on a GB300 (2048 rows over 16384 keys).  24/4 heads of
// 256: 499 us, 1760 TFLOP/s, 0.90 of the dense peak; a tile's products want 2048
// cycles and take about 2600, because Q K^T with both operands in shared memory
// reads 128 bytes a cycle, all that shared memory gives, beside the tile copies.
// With a cap 600 us: the polynomial makes the softmax of a tile (3700 cycles) the
// longest part of the S -> W -> O chain, of which two are in flight.  32/8 heads of
// 128: 409 us, 1430 TFLOP/s: the chain again, 1024 cycles of exponentials (16 a
// cycle) for 1024 cycles of products.  Tried and dropped: exponentials of one pair
// in four by a polynomial (FMA issue was the next limit: 520 against then 462 us at
// head_dim 128), and the maximum, the scores and the weights in one pass that is
// repeated when the maximum moves (its branches keep the compiler from overlapping
// the 32-column steps: 594 against then 550 us at 256, 592 against 442 us at 128).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace i8kv {
namespace bp {

constexpr int kBS = 16;
constexpr int kRows = 128;          // rows of one MMA: one per tensor-memory lane
__host__ __device__ constexpr bool paired(int D) { return D <= 128; }
__host__ __device__ constexpr int block_rows(int D) { return paired(D) ? 2 * kRows : kRows; }
constexpr int kKeys = 128;
constexpr int kBlk = kKeys / kBS;  // cache blocks per tile
constexpr int kThreads = 384;
constexpr int kWG = 128;
constexpr int kSoftWarp = 4;
constexpr float kLazy = 8.0f;
// Registers: 128 control threads at 40, 256 softmax threads at 232 (128 scores
// each); 40 + 2 x 232 = 3 x 168, what 384 threads launch with.
constexpr int kRegsCtl = 40, kRegsSoft = 232;
static_assert(kRegsCtl + 2 * kRegsSoft <= 3 * 168, "register split");
constexpr int kSnap = 2;
constexpr int kScales = 3 * kBlk;  // per tile: sK, log2 sV, 1 / sV of its blocks

// The workspace (all offsets multiples of 128 bytes): where every CTA's range
// starts (cuts [grid + 1] and a header each), the row blocks' ranges, the operand
// tiles and their scales, the records.
struct Head {
  int rb, kvh, first, cnt;  // row block, KV head, tiles of the row block before the range, its tiles
};
struct Range {
  int lo, hi;        // the row block's tiles
  int lo_in, hi_in;  // keys that every row of it sees
};
struct Plan {
  int nrb, tile0, ntiles, grid;
  size_t oCuts, oHead, oRange, oScale, oK, oV, oRec, bytes;
};
inline Plan plan_of(int H, int C, int G, int Hkv, int D, int window, int grid) {
  Plan p;
  auto up = [](size_t x) { return (x + 127) / 128 * 128; };
  const int rows = block_rows(D);
  p.nrb = (int)(((int64_t)C * G + rows - 1) / rows);
  p.tile0 = window > 0 && H - window + 1 > 0 ? (H - window + 1) / kKeys : 0;  // no row sees an earlier key
  p.ntiles = (H + C + kKeys - 1) / kKeys - p.tile0;
  p.grid = grid;
  const size_t tile = (size_t)kKeys * D * 2, n = (size_t)p.ntiles * Hkv;
  p.oCuts = 0;
  p.oHead = up(sizeof(int) * ((size_t)grid + 1));
  p.oRange = p.oHead + up(sizeof(Head) * (size_t)grid);
  p.oScale = p.oRange + up(sizeof(Range) * (size_t)p.nrb);
  p.oK = p.oScale + up(n * kScales * 4);
  p.oV = p.oK + n * tile;
  p.oRec = p.oV + n * tile;
  p.bytes = p.oRec + (size_t)2 * grid * rows * (D + 2) * 4;
  return p;
}

struct Params {
  BlockDecodeParams a;
  Plan w;
};

template <int D>
struct Lay {
  static constexpr bool kPair = paired(D);
  static constexpr int kRB = block_rows(D);            // rows of a row block
  static constexpr int kParts = D == 256 ? 2 : 1;      // stages per operand tile
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kStage = kTile / kParts;        // two parts: K half the dims, V half the keys
  static constexpr int kStages = D == 64 ? 11 : 5;
  static constexpr int kQ = kRB * D * 2;
  static constexpr int oQ = 0;                         // [kRB / 128][D/64][128 rows][128 B]
  static constexpr int oRing = oQ + kQ;
  static constexpr int oM = oRing + kStages * kStage;  // M [2][128]
  static constexpr int oL = oM + 2 * kRows * 4;        // the warpgroups' row sums [2][128]
  static constexpr int oSc = oL + 2 * kRows * 4;       // scales of kSc tiles
  static constexpr int kSc = D == 64 ? 8 : 4;          // a slot is refilled only after its tile's products
  static constexpr int oBar = oSc + kSc * kScales * 4;
  // full[kStages], free[kStages], sc_full[kSc], s_full[2], p_full[2][2], m_full[2], pv_done[2], q_full[2], o_free[2]
  static constexpr int kBars = 2 * kStages + kSc + 2 + 4 + 2 + 2 + 2 + 2;
  static constexpr int oCtl = oBar + kBars * 8;
  static constexpr int kTotal = oCtl + 16;
  static_assert(kTotal <= 232448, "shared memory");
  static constexpr uint32_t kOCol = 256;  // O; in pairs the second one D columns on
};

// Byte offset of 16-byte chunk c of row r of a 128-byte-row tile, swizzled.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ void interval(const BlockDecodeParams& p, int j, int& lo, int& hi) {
  lo = 0;
  if (p.window > 0) lo = max(0, p.H + j - p.window + 1);
  if (p.key_begin != nullptr) lo = max(lo, p.key_begin[j]);
  hi = p.H + j + 1;
  if (p.key_end != nullptr) hi = max(0, min(p.key_end[j], p.H + p.C));
}

__device__ __forceinline__ uint32_t bf16x2_codes(uint32_t w, int i) {
  return bf16x2_rn((float)(int8_t)((w >> (8 * i)) & 0xffu), (float)(int8_t)((w >> (8 * i + 8)) & 0xffu));
}

// Chunks 2 q and 2 q + 1 of a row of swizzled 128-byte rows: one 32-byte sector,
// written whole where the workspace allows it.  By halves it is two partial writes:
// 18432 keys, 4 KV heads of 256: 18.3 us, 6.2 TB/s read and written, against 30.
__device__ __forceinline__ void put_pair(uint8_t* rows, int row, int q, uint4 a, uint4 b, bool wide) {
  if (wide) {
    if (row & 1) {
      const uint4 t = a;
      a = b;
      b = t;
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(rows + (swz(row, 2 * q) & ~16u)), "r"(a.x),
                 "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(rows + swz(row, 2 * q)) = a;
    *reinterpret_cast<uint4*>(rows + swz(row, 2 * q + 1)) = b;
  }
}


// ---- operand tiles and scales: one CTA per (tile, KV head) for the keys and one
// for the values; also the row blocks' tile ranges, spread over the latter's warps.
template <int D>
__global__ void __launch_bounds__(256) block_tiles_kernel(const __grid_constant__ Params pp) {
  const BlockDecodeParams& p = pp.a;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x, kvh = blockIdx.y;
  const bool keys = blockIdx.z == 0;
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  // row block ranges
  for (int rb = keys ? pp.w.nrb : (blockIdx.y * gridDim.x + blockIdx.x) * 8 + warp; rb < pp.w.nrb; rb += gridDim.x * gridDim.y * 8) {
    constexpr int kRB = block_rows(D);
    const int j0 = p.divG.div(rb * kRB), j1 = min(p.C - 1, p.divG.div(rb * kRB + kRB - 1));
    int lo = 0x7fffffff, hi = 0, lo_in = 0, hi_in = 0x7fffffff;
    for (int j = j0 + lane; j <= j1; j += 32) {
      int a, b;
      interval(p, j, a, b);
      lo_in = max(lo_in, a);
      hi_in = min(hi_in, b);
      if (a < b) {
        lo = min(lo, a);
        hi = max(hi, b);
      }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    lo_in = __reduce_max_sync(0xffffffffu, lo_in);
    hi_in = __reduce_min_sync(0xffffffffu, hi_in);
    if (lane == 0) {
      Range r;
      r.lo = lo < hi ? lo / kKeys : 0;
      r.hi = lo < hi ? (hi + kKeys - 1) / kKeys : 0;
      r.lo_in = lo_in;
      r.hi_in = hi_in;
      reinterpret_cast<Range*>(ws + pp.w.oRange)[rb] = r;
    }
  }
  const int n = p.H + p.C;
  const int blk0 = (pp.w.tile0 + tile) * kBlk;
  int phys[kBlk];
#pragma unroll
  for (int i = 0; i < kBlk; ++i) {
    phys[i] = -1;
    if ((blk0 + i) * kBS < n) {
      const int b = __ldg(p.block_tables + blk0 + i);
      phys[i] = b >= 0 && b < p.num_blocks ? b : -2;  // -2: no such block; an error for a row that sees it
    }
  }
  const size_t ti = (size_t)kvh * pp.w.ntiles + tile;
  uint8_t* kt = ws + pp.w.oK + ti * Lay<D>::kTile;
  uint8_t* vt = ws + pp.w.oV + ti * Lay<D>::kTile;
  if (keys && tid < kBlk) {
    float sk = 0.f, sv = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kBlk; ++i)
      if (i == tid) {
        bad = phys[i] == -2;
        if (phys[i] >= 0) {
          sk = p.k_scale[(size_t)phys[i] * p.Hkv + kvh] * p.score_mul;
          sv = p.v_scale[(size_t)phys[i] * p.Hkv + kvh];
        }
      }
    sv = fmaxf(sv, kTinyDivisor);
    float* s = reinterpret_cast<float*>(ws + pp.w.oScale) + ti * kScales;
    s[tid] = sk;
    s[kBlk + tid] = bad ? 0.f : log2f(sv);
    s[2 * kBlk + tid] = bad ? -1.f : __frcp_rn(sv);
  }
  // K page [D/16][16 tokens][16 B] and V page [D][16 B]: D chunks each per block.
  // D = 256: a thread per chunk; below, 256 / D blocks at once.
  constexpr int kAt = 256 / D, kIn = kBlk / kAt;
  const bool wide = (reinterpret_cast<uintptr_t>(ws) & 31) == 0;
  const int sub = tid / D, c = tid % D;
#pragma unroll
  for (int i0 = 0; i0 < kBlk; i0 += kIn * kAt) {
    uint4 x[kIn];
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      int ph = -1;
#pragma unroll
      for (int s = 0; s < kAt; ++s)
        if (i0 + u * kAt + s < kBlk && s == sub) ph = phys[(i0 + u * kAt + s) % kBlk];
      x[u] = make_uint4(0, 0, 0, 0);
      if (ph >= 0)
        x[u] = __ldg(reinterpret_cast<const uint4*>((keys ? p.k_cache : p.v_cache) + ((size_t)ph * p.Hkv + kvh) * (D * kBS)) + c);
    }
#pragma unroll
    for (int u = 0; u < kIn; ++u) {
      const int i = i0 + u * kAt + sub;
      uint4 h0, h1;
      if (keys) {
        const int dc = c / kBS, key = i * kBS + c % kBS;
        h0 = make_uint4(bf16x2_codes(x[u].x, 0), bf16x2_codes(x[u].x, 2), bf16x2_codes(x[u].y, 0), bf16x2_codes(x[u].y, 2));
        h1 = make_uint4(bf16x2_codes(x[u].z, 0), bf16x2_codes(x[u].z, 2), bf16x2_codes(x[u].w, 0), bf16x2_codes(x[u].w, 2));
        put_pair(kt + (size_t)(dc / 4) * (kKeys * 128), key, dc % 4, h0, h1, wide);
      } else {
        s8x4_to_f16(x[u].x, h0.x, h0.y);
        s8x4_to_f16(x[u].y, h0.z, h0.w);
        s8x4_to_f16(x[u].z, h1.x, h1.y);
        s8x4_to_f16(x[u].w, h1.z, h1.w);
        put_pair(vt + (size_t)(i / 4) * (D * 128), c, i % 4, h0, h1, wide);
      }
    }
  }
}

// A value that is the same in every lane, known as such to the compiler.
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// ---- the walk over a CTA's range of the list (KV head, row block, tile)
struct Walk {
  int kvh, rb, first, len, left, cnt, lo;  // segment: tiles lo + first .. + len of the row block
};
__device__ __forceinline__ void walk_load(const Range* rg, Walk& w) {
  w.lo = uni(rg[w.rb].lo);
  w.cnt = uni(rg[w.rb].hi) - w.lo;
  w.len = min(w.cnt - w.first, w.left);
}
__device__ __forceinline__ bool walk_next(const Params& pp, const Range* rg, Walk& w) {
  w.left -= w.len;
  if (w.left <= 0) return false;
  w.first = 0;
  do {
    if (++w.rb == pp.w.nrb) {
      w.rb = 0;
      if (++w.kvh == pp.a.Hkv) return false;
    }
    walk_load(rg, w);
  } while (w.cnt == 0);
  return true;
}

// The cut of the list over the CTAs: `per` steps each, the first `rem` one more.
__device__ __forceinline__ int cut_at(int per, int rem, int c) { return per * c + min(c, rem); }

// Bounded wait that gives up at once when the CTA has aborted (error 1 after the
// time limit); every thread still runs its loops and barriers.
__device__ __forceinline__ void pwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return;
  if (*abort_flag) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      record_error(1);
      *abort_flag = 1;
      return;
    }
  }
}
// The same for a whole warp that stays together; false once the CTA has aborted.
__device__ __forceinline__ bool pwait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  pwait(bar, parity, abort_flag);
  return !__any_sync(0xffffffffu, *abort_flag != 0);
}
// One lane of a converged warp.  The copies and MMAs are issued under it by a
// warp whose control flow is uniform, so their operands live in uniform
// registers: issued by "lane 0" of a divergent branch each MMA took about 150
// cycles to hand over, longer than it runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// 16-byte units of 32 rows: lane i of a group of U lanes holds units 0 .. U - 1 of
// row i of the group; afterwards unit i of its rows 0 .. U - 1.
template <int U>
__device__ __forceinline__ void transpose_units(uint4 (&u)[U], int lane) {
#pragma unroll
  for (int s = 1; s < U; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (k & s) continue;
      uint4 send = up ? u[k] : u[k | s], got;
      got.x = __shfl_xor_sync(0xffffffffu, send.x, s);
      got.y = __shfl_xor_sync(0xffffffffu, send.y, s);
      got.z = __shfl_xor_sync(0xffffffffu, send.z, s);
      got.w = __shfl_xor_sync(0xffffffffu, send.w, s);
      if (up) u[k] = got;
      else u[k | s] = got;
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The part of (a, b) that their packed f16 `hi` leaves over, as f16x2.
__device__ __forceinline__ uint32_t f16x2_rest(uint32_t hi, float a, float b) {
  float fa, fb;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(fa), "=f"(fb) : "r"(hi));
  return f16x2_of(a - fa, b - fb);
}

template <int D, bool kCap, bool kSlope, bool kHiLo>
__global__ void __launch_bounds__(kThreads, 1) block_prefix_kernel(const __grid_constant__ Params pp) {
  using Ly = Lay<D>;
  constexpr int NS = Ly::kStages;
  const BlockDecodeParams& p = pp.a;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly::oBar);
  uint64_t* free_ = full + NS;
  uint64_t* sc_full = free_ + NS;   // [n % kSc] scales of tile n
  // per S slot (in pairs the warpgroup, else n & 1):
  uint64_t* s_full = sc_full + Ly::kSc;  // S in tensor memory
  uint64_t* p_full = s_full + 2;    // W in tensor memory: [slot][keys 0..63, 64..127]
  uint64_t* m_full = p_full + 4;    // the running maxima after the tile (not in pairs)
  uint64_t* pv_done = m_full + 2;   // its product has joined O
  uint64_t* q_full = pv_done + 2;   // the segment's query rows in shared memory (in pairs one per warpgroup)
  uint64_t* o_free = q_full + 2;    // the segment's O is read (in pairs one per warpgroup)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Ly::oCtl);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::oCtl + 4);
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const Range* rg = reinterpret_cast<const Range*>(ws + pp.w.oRange);

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&free_[i], 1);
    }
    for (int i = 0; i < Ly::kSc; ++i) mbar_init(&sc_full[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], kWG);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&m_full[i], kWG);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kWG);
      mbar_init(&o_free[i], Ly::kPair ? kWG : 2 * kWG);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of the list ----
  int* scan = reinterpret_cast<int*>(smem + Ly::oQ);  // [12] warp sums, [16 ..] the start
  const int grid = gridDim.x;
  auto scan_step = [&](int v, int& before) {
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int base = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) base += scan[i];
      sum += scan[i];
    }
    before = base + x - v;
    return sum;
  };
  int per_head = 0, before;
  for (int r0 = 0; r0 < pp.w.nrb; r0 += kThreads) {
    const int rb = r0 + tid;
    per_head += scan_step(rb < pp.w.nrb ? rg[rb].hi - rg[rb].lo : 0, before);
  }
  const int total = per_head * p.Hkv;
  const int per = p.divGrid.div(total), rem = total - per * grid;
  int u[2], kvh[2];  // the range's ends: place in the list, KV head
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    u[e] = cut_at(per, rem, blockIdx.x + e);
    kvh[e] = u[e] < total ? u[e] / per_head : 0;
  }
  if (tid < 6) scan[16 + tid] = 0;  // row block, tile in it, its tiles
  {
    int run = 0;
    for (int r0 = 0; r0 < pp.w.nrb; r0 += kThreads) {
      const int rb = r0 + tid;
      const int cnt = rb < pp.w.nrb ? rg[rb].hi - rg[rb].lo : 0;
      const int sum = scan_step(cnt, before);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int in = u[e] - kvh[e] * per_head - (run + before);
        if (u[e] < total && in >= 0 && in < cnt) {
          scan[16 + 3 * e] = rb;
          scan[17 + 3 * e] = in;
          scan[18 + 3 * e] = cnt;
        }
      }
      run += sum;
    }
  }
  __syncthreads();
  // A cut near the border of two row blocks moves there, by up to kSnap tiles: a
  // segment more costs its CTA about as much, and its record is written and merged.
  Walk w;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int in = scan[17 + 3 * e], cnt = scan[18 + 3 * e], reach = min(kSnap, (per + 1) / 2);
    int first = in;
    if (u[e] > 0 && u[e] < total) {
      if (in <= reach) first = 0;
      else if (cnt - in <= reach) first = cnt;
    }
    u[e] = uni(u[e] + first - in);
    if (e == 0) {
      w.rb = uni(scan[16]);
      w.first = uni(first);
    }
  }
  const int u0 = u[0], u1 = u[1];
  int* cuts = reinterpret_cast<int*>(ws + pp.w.oCuts);
  if (tid == 0) {
    cuts[blockIdx.x] = u0;
    if (blockIdx.x + 1 == gridDim.x) cuts[gridDim.x] = u1;
  }
  w.kvh = uni(kvh[0]);
  w.left = u1 - u0;
  walk_load(rg, w);
  if (w.left > 0 && w.len == 0) walk_next(pp, rg, w);  // the range starts with the next row block
  if (tid == 0) reinterpret_cast<Head*>(ws + pp.w.oHead)[blockIdx.x] = Head{w.rb, w.kvh, w.first, w.cnt};
  // row blocks without a visible key: zero rows
  for (int rb = blockIdx.x; rb < pp.w.nrb; rb += grid) {
    if (rg[rb].hi != rg[rb].lo) continue;
    for (int i = tid; i < Ly::kRB * (D / 4); i += kThreads) {
      const int64_t r = (int64_t)rb * Ly::kRB + i / (D / 4);
      if (r < (int64_t)p.C * p.G)
        for (int k = 0; k < p.Hkv; ++k)
          store_out4(p.out, p.out_bf16, ((size_t)(r / p.G) * p.Hq + k * p.G + r % p.G) * D + (i % (D / 4)) * 4,
                     make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  __syncthreads();  // the scan buffer (the query tile) is free

  if (warp < kSoftWarp) {
    regs_dec<kRegsCtl>();
    if (u0 < u1 && warp == 0) {
      // ================= tile copies =================
      int st = 0, lap = 0, c = 0, n = 0;  // next stage, laps of the ring; stages filled, tiles of K
      const uint8_t* src[2] = {ws + pp.w.oK, ws + pp.w.oV};
      const float* scl = reinterpret_cast<const float*>(ws + pp.w.oScale);
      bool ok = true;
      auto load = [&](int which, size_t ti) {
#pragma unroll
        for (int h = 0; h < Ly::kParts; ++h) {
          if (ok && lap > 0) ok = pwait_warp(&free_[st], (lap - 1) & 1, abort_flag);
          if (!ok) return;
          if (elect_one()) {
            mbar_expect_tx(&full[st], Ly::kStage);
            bulk_g2s(smem + Ly::oRing + st * Ly::kStage, src[which] + ti * Ly::kTile + h * Ly::kStage, Ly::kStage, &full[st]);
            mbar_arrive(&full[st]);
            if (which == 0 && h == 0) {
              uint64_t* b = &sc_full[n % Ly::kSc];
              mbar_expect_tx(b, kScales * 4);
              bulk_g2s(smem + Ly::oSc + (n % Ly::kSc) * kScales * 4, scl + ti * kScales, kScales * 4, b);
              mbar_arrive(b);
            }
          }
          __syncwarp();
          ++c;
          if (++st == NS) {
            st = 0;
            ++lap;
          }
        }
        n += which == 0;
      };
      do {
        const size_t t0 = (size_t)w.kvh * pp.w.ntiles + (w.lo + w.first - pp.w.tile0);
        load(0, t0);
        for (int t = 0; t < w.len && ok; ++t) {  // in the order of their use
          if (Ly::kPair) load(1, t0 + t);
          if (t + 1 < w.len) load(0, t0 + t + 1);
          if (!Ly::kPair) load(1, t0 + t);
        }
      } while (ok && walk_next(pp, rg, w));
      if (!ok) {  // copies under way land before the CTA exits
        for (int k = max(0, c - NS); k < c; ++k) mbar_wait(&full[k % NS], (k / NS) & 1);
        for (int k = max(0, n + 1 - Ly::kSc); k <= n; ++k) mbar_wait(&sc_full[k % Ly::kSc], (k / Ly::kSc) & 1);
      }
    } else if (u0 < u1 && warp == 1) {
      // ================= MMA issue =================
      constexpr uint32_t idesc_qk = umma_idesc_bf16(kRows, kKeys);
      constexpr uint32_t idesc_pv = umma_idesc_f16(kRows, D);
      const uint64_t qdesc = umma_desc(smem_u32(smem + Ly::oQ), 128), rdesc = umma_desc(smem_u32(smem + Ly::oRing), 128);
      int st = 0, lap = 0, n = 0, seg = 0;
      uint64_t* last = nullptr;
      uint32_t last_par = 0;
      bool ok = true;
      auto next_stage = [&]() {
        if (++st == NS) {
          st = 0;
          ++lap;
        }
      };
      // a K = 16 step is 32 bytes of a 128-byte row; the descriptors count 16-byte units
      if constexpr (Ly::kPair) {
        // S of rows 128 g .. + 127 of the row block from the K stage at kd, and O += W V
        auto qk_half = [&](int g, uint64_t kd) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_f16(tmem + g * kKeys, qdesc + g * (kRows * D / 8) + (k / 4) * (kRows * 8) + (k % 4) * 2,
                     kd + (k / 4) * (kKeys * 8) + (k % 4) * 2, idesc_qk, k > 0);
          umma_commit(&s_full[g]);
        };
        auto pv_half = [&](int g, int half, uint64_t vd, bool add) {  // the tile's keys 64 half .. + 63
#pragma unroll
          for (int k = 4 * half; k < 4 * half + 4; ++k) {
            const uint64_t b = vd + (k / 4) * (D * 8) + (k % 4) * 2;
            umma_f16_ta(tmem + Ly::kOCol + g * D, tmem + g * kKeys + k * 8, b, idesc_pv, add || k > 0);
            if constexpr (kHiLo) umma_f16_ta(tmem + Ly::kOCol + g * D, tmem + g * kKeys + 64 + k * 8, b, idesc_pv, true);
          }
          if (half) umma_commit(&pv_done[g]);
        };
        int n2 = 0, seg2 = 0;  // tiles and segments of the second warpgroup
        do {
          const bool two = w.rb * Ly::kRB + kRows < p.C * p.G;
          ok = pwait_warp(&q_full[0], seg & 1, abort_flag) && (!two || pwait_warp(&q_full[1], seg2 & 1, abort_flag)) &&
               pwait_warp(&full[st], lap & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t kd = rdesc + (uint64_t)(st * (Ly::kStage / 16));
            qk_half(0, kd);
            if (two) qk_half(1, kd);
            umma_commit(&free_[st]);
          }
          __syncwarp();
          next_stage();
          for (int t = 0; t < w.len; ++t) {
            const bool more = t + 1 < w.len;
            const int vs = st, ks = st + 1 == NS ? 0 : st + 1, klap = st + 1 == NS ? lap + 1 : lap;
            const uint64_t vd = rdesc + (uint64_t)(vs * (Ly::kStage / 16)), kd = rdesc + (uint64_t)(ks * (Ly::kStage / 16));
            ok = pwait_warp(&full[vs], lap & 1, abort_flag) && (!more || pwait_warp(&full[ks], klap & 1, abort_flag)) &&
                 (t > 0 || seg == 0 || pwait_warp(&o_free[0], (seg - 1) & 1, abort_flag)) &&
                 pwait_warp(&p_full[0], n & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) pv_half(0, 0, vd, t > 0);
            __syncwarp();
            ok = pwait_warp(&p_full[1], n & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              pv_half(0, 1, vd, true);
              if (more) qk_half(0, kd);
            }
            __syncwarp();
            if (two) {
              ok = (t > 0 || seg2 == 0 || pwait_warp(&o_free[1], (seg2 - 1) & 1, abort_flag)) &&
                   pwait_warp(&p_full[2], n2 & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
              if (elect_one()) pv_half(1, 0, vd, t > 0);
              __syncwarp();
              ok = pwait_warp(&p_full[3], n2 & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
            }
            if (elect_one()) {
              if (two) pv_half(1, 1, vd, true);
              umma_commit(&free_[vs]);
              if (more) {
                if (two) qk_half(1, kd);
                umma_commit(&free_[ks]);
              }
              last = &free_[more ? ks : vs];
              last_par = (more ? klap : lap) & 1;
            }
            __syncwarp();
            next_stage();
            if (more) next_stage();
            ++n;
            n2 += two;
          }
          ++seg;
          seg2 += two;
        } while (ok && walk_next(pp, rg, w));
      } else {
      auto qk = [&](int m) {  // S of the CTA's tile m
#pragma unroll
        for (int h = 0; h < Ly::kParts; ++h) {
          if (ok) ok = pwait_warp(&full[st], lap & 1, abort_flag);
          if (!ok) return;
          tc_fence_after();
          constexpr int kSteps = D / 16 / Ly::kParts;
          const uint64_t kd = rdesc + (uint64_t)(st * (Ly::kStage / 16));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const int kk = h * kSteps + k;
              umma_f16(tmem + (m & 1) * kKeys, qdesc + (kk / 4) * (kRows * 8) + (kk % 4) * 2,
                       kd + (k / 4) * (kKeys * 8) + (k % 4) * 2, idesc_qk, kk > 0);
            }
            umma_commit(&free_[st]);
            if (h == Ly::kParts - 1) umma_commit(&s_full[m & 1]);
          }
          __syncwarp();
          next_stage();
        }
        last = &s_full[m & 1];
        last_par = (m >> 1) & 1;
      };
      do {
        ok = pwait_warp(&q_full[0], seg & 1, abort_flag);
        if (ok) qk(n);
        for (int t = 0; t < w.len && ok; ++t, ++n) {
          if (t + 1 < w.len) qk(n + 1);
          if (ok && t == 0 && seg > 0) ok = pwait_warp(&o_free[0], (seg - 1) & 1, abort_flag);
#pragma unroll
          for (int h = 0; h < Ly::kParts; ++h) {  // the two halves of the keys, as their weights arrive
            if (ok) ok = pwait_warp(&full[st], lap & 1, abort_flag);
            if (ok) ok = pwait_warp(&p_full[2 * (n & 1) + h], (n >> 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            constexpr int kSteps = kKeys / 16 / Ly::kParts;
            const uint64_t vd = rdesc + (uint64_t)(st * (Ly::kStage / 16));
            const uint32_t wt = tmem + (n & 1) * kKeys;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                const int kk = h * kSteps + k;
                const uint64_t b = vd + (k / 4) * (D * 8) + (k % 4) * 2;
                umma_f16_ta(tmem + Ly::kOCol, wt + kk * 8, b, idesc_pv, t > 0 || kk > 0);
                if constexpr (kHiLo) umma_f16_ta(tmem + Ly::kOCol, wt + 64 + kk * 8, b, idesc_pv, true);
              }
              umma_commit(&free_[st]);
              if (h == Ly::kParts - 1) umma_commit(&pv_done[n & 1]);
            }
            __syncwarp();
            next_stage();
          }
          if (ok) {
            last = &pv_done[n & 1];
            last_par = (n >> 1) & 1;
          }
        }
        ++seg;
      } while (ok && walk_next(pp, rg, w));
      }
      if (last) mbar_wait(last, last_par);  // every MMA has completed before tensor memory is released
    }
    __syncwarp();
  } else {
    // ================= softmax: a thread per row =================
    // In pairs each warpgroup has 128 rows, a slot of S and an O of its own and takes
    // every tile; else both have the same rows and take alternate tiles.
    regs_inc<kRegsSoft>();
    const int wg = (warp - kSoftWarp) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to0 = trow + Ly::kOCol + (Ly::kPair ? wg * D : 0);  // this row of O
    float* mref = reinterpret_cast<float*>(smem + Ly::oM);
    float* lrow = reinterpret_cast<float*>(smem + Ly::oL);
    const int R = p.C * p.G;
    // The query rows of a segment's row block (in pairs of this warpgroup's half):
    // whole rows by neighbouring lanes, asked for as soon as the previous segment's
    // last S is complete, that is, once its products have read the old rows.
    auto ask_q = [&](const Walk& x) {
      constexpr int kLanes = D / 8, kAt = kWG / kLanes;  // threads per row, rows at once
      const int c = (tid & (kWG - 1)) % kLanes, row0 = (tid & (kWG - 1)) / kLanes;
      const int r0 = x.rb * Ly::kRB + (Ly::kPair ? wg * kRows : 0) + row0;
      uint8_t* dst = smem + Ly::oQ + (Ly::kPair ? wg * (kRows * D * 2) : 0) + (c / 8) * (kRows * 128);
#pragma unroll 4
      for (int i = 0; i < kRows; i += kAt) {
        const int r = r0 + i, j = p.divG.div(r), h = r - j * p.G;
        const bool in = r < R;
        const uint16_t* src = p.q + (in ? (int64_t)j * p.q_stride + (size_t)(x.kvh * p.G + h) * D + c * 8 : 0);
        cp_async_16(dst + swz(row0 + i, c % 8), src, in ? 16u : 0u);
      }
    };
    auto hand_q = [&]() {
      cp_async_wait_all();
      fence_async_smem();
      mbar_arrive(&q_full[Ly::kPair ? wg : 0]);
    };
    auto has_rows = [&](const Walk& x) { return !Ly::kPair || x.rb * Ly::kRB + wg * kRows < R; };
    int n = 0, tile = 0;  // this warpgroup's tiles in pairs, else the CTA's; the CTA's
    bool first_seg = true, more = u0 < u1;
    if (more && has_rows(w) && (Ly::kPair || wg == 0)) {
      ask_q(w);
      hand_q();
    }
    while (more) {
      Walk next = w;
      more = walk_next(pp, rg, next);
      if (!has_rows(w)) {  // the last row block may have rows for one warpgroup only
        if (more && has_rows(next)) {
          ask_q(next);
          hand_q();
        }
        tile += w.len;
        first_seg = false;
        w = next;
        continue;
      }
      const int r = w.rb * Ly::kRB + (Ly::kPair ? wg * kRows : 0) + row;
      const bool valid = r < R;
      const int j = valid ? p.divG.div(r) : 0, hq = w.kvh * p.G + (valid ? r - j * p.G : 0);
      int lo = 0, hi = 0;
      if (valid) interval(p, j, lo, hi);
      const int pos = p.H + j;
      float slope = 0.f;
      if constexpr (kSlope) slope = valid ? -__ldg(p.slopes + hq) * kLog2e : 0.f;
      bool asked = false;
      float l = 0.f, Mown = -INFINITY;
      for (int t = 0; t < w.len; ++t, ++n, ++tile) {
        if (!Ly::kPair && (n & 1) != wg) continue;
        const int key0 = (w.lo + w.first + t) * kKeys;
        const int slot = Ly::kPair ? wg : n & 1, phase = Ly::kPair ? n & 1 : (n >> 1) & 1;
        pwait(&s_full[slot], phase, abort_flag);
        pwait(&sc_full[tile % Ly::kSc], (tile / Ly::kSc) & 1, abort_flag);  // landed before S
        if (t + 1 == w.len && more && has_rows(next)) {
          ask_q(next);
          asked = true;
        }
        const float* sc = reinterpret_cast<const float*>(smem + Ly::oSc) + (tile % Ly::kSc) * kScales;
        __syncwarp();
        tc_fence_after();
        const uint32_t ts = trow + slot * kKeys;
        float v[kKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, *reinterpret_cast<float(*)[32]>(v + 32 * c));
        tmem_wait_ld();
        // the block's addend of offset i: log2 sV, and with a bias slope (pos - key)
        auto addend = [&](int b, int i) {
          float base = sc[kBlk + b];
          if constexpr (kSlope)
            base = __fmaf_rn(-slope, (float)i, __fmaf_rn(slope, (float)(pos - key0 - b * kBS), base));
          return base;
        };
        // u = score log2 e (+ bias) + log2 sV
        if constexpr (kCap) {
          // z = score / cap; cap log2 e tanh z = z P(z^2), on the FMA pipes that the
          // exponentials leave idle: P interpolates tanh(z) / z at Chebyshev nodes, of
          // degree 2 for |z| <= 1/4 and 3 for |z| <= 1/2 (4e-7 and 6e-7 relative; bf16
          // outputs) or 6 for |z| <= 1 (5e-8)
          float zmax = 0.f;
#pragma unroll
          for (int b = 0; b < kBlk; ++b) {
            const uint64_t ks2 = f2(sc[b], sc[b]);
#pragma unroll
            for (int i = b * kBS; i < (b + 1) * kBS; i += 2) {
              f2_split(mul2(f2(v[i], v[i + 1]), ks2), v[i], v[i + 1]);
              zmax = max3(zmax, fabsf(v[i]), fabsf(v[i + 1]));
            }
          }
          auto poly = [&](auto deg, const float* coef) {
            constexpr int N = decltype(deg)::value;
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
#pragma unroll
              for (int i = b * kBS; i < (b + 1) * kBS; i += 2) {
                const uint64_t z = f2(v[i], v[i + 1]), y = mul2(z, z);
                uint64_t a = f2(coef[N], coef[N]);
#pragma unroll
                for (int d = N - 1; d >= 0; --d) a = fma2(a, y, f2(coef[d], coef[d]));
                f2_split(fma2(a, z, f2(addend(b, i - b * kBS), addend(b, i + 1 - b * kBS))), v[i], v[i + 1]);
              }
          };
          if (!kHiLo && __all_sync(0xffffffffu, zmax <= 0.25f)) {
            poly(std::integral_constant<int, 2>{}, p.cap_poly2);
          } else if (!kHiLo && __all_sync(0xffffffffu, zmax <= 0.5f)) {
            poly(std::integral_constant<int, 3>{}, p.cap_poly3);
          } else if (__all_sync(0xffffffffu, zmax <= 1.f)) {
            poly(std::integral_constant<int, kCapDeg>{}, p.cap_poly);
          } else {  // some score above the cap: 1 - 2 / (e^2z + 1)
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
#pragma unroll
              for (int i = b * kBS; i < (b + 1) * kBS; ++i)
                v[i] = __fmaf_rn(-2.f * p.cap_log2, rcp_approx(ex2(v[i] * (2.f * kLog2e)) + 1.f),
                                 p.cap_log2 + addend(b, i - b * kBS));
          }
        } else {
#pragma unroll
          for (int b = 0; b < kBlk; ++b) {
            const uint64_t ks2 = f2(sc[b], sc[b]);
#pragma unroll
            for (int i = b * kBS; i < (b + 1) * kBS; i += 2)
              f2_split(fma2(f2(v[i], v[i + 1]), ks2, f2(addend(b, i - b * kBS), addend(b, i + 1 - b * kBS))), v[i], v[i + 1]);
          }
        }
        if constexpr (kSlope) {  // keys behind the row: |pos - t|, the linear form has the other sign
          if (__any_sync(0xffffffffu, key0 + kKeys - 1 > pos && hi > pos + 1)) {
            const float d0 = (float)(key0 - pos);
#pragma unroll
            for (int i = 0; i < kKeys; ++i) v[i] = __fmaf_rn(2.f * slope, fmaxf(d0 + (float)i, 0.f), v[i]);
          }
        }
        // hidden keys: only blocks of 16 in which some row of the warp has any
        if (!__all_sync(0xffffffffu, key0 >= lo && key0 + kKeys <= hi)) {
          const int a = lo - key0, e = hi - key0;
#pragma unroll
          for (int b = 0; b < kBlk; ++b)
            if (__any_sync(0xffffffffu, a > b * kBS || e < (b + 1) * kBS)) {
#pragma unroll
              for (int i = b * kBS; i < (b + 1) * kBS; ++i) v[i] = i >= a && i < e ? v[i] : -INFINITY;
            }
        }
        float mb[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          mb[b] = max3(v[b * 16], v[b * 16 + 1], v[b * 16 + 2]);
#pragma unroll
          for (int i = 3; i + 1 < 16; i += 2) mb[b] = max3(mb[b], v[b * 16 + i], v[b * 16 + i + 1]);
          mb[b] = fmaxf(mb[b], v[b * 16 + 15]);
        }
        const float mx = fmaxf(max3(max3(mb[0], mb[1], mb[2]), mb[3], mb[4]), max3(mb[5], mb[6], mb[7]));
        // the running maximum: this thread's own in pairs, else from the neighbour's
        // tile and on to the neighbour's next
        float M = Ly::kPair ? Mown : -INFINITY;
        if (!Ly::kPair && t > 0) {
          pwait(&m_full[(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag);
          M = mref[((n - 1) & 1) * kRows + row];
        }
        float alpha = 1.f;
        if (mx > M + kLazy || M == -INFINITY) {
          if (M != -INFINITY) alpha = ex2(M - mx);
          M = mx;
        }
        if constexpr (!Ly::kPair) {
          mref[(n & 1) * kRows + row] = M;
          mbar_arrive(&m_full[n & 1]);
        }
        const float m0 = M == -INFINITY ? 0.f : M;  // a row that has seen no key yet
        if (Mown != M) {
          l = Mown == -INFINITY ? 0.f : l * ex2(Mown - M);
          Mown = M;
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, alpha != 1.f)) {  // rare: O joins the new maximum
          pwait(&pv_done[Ly::kPair ? wg : (n - 1) & 1], Ly::kPair ? (n - 1) & 1 : ((n - 1) >> 1) & 1, abort_flag);
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            uint32_t ob[32];
            tmem_ld32(to0 + 32 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) ob[i] = __float_as_uint(o[i] * alpha);
            tmem_st32(to0 + 32 * c, ob);
          }
        }
        const uint64_t nm = f2(-m0, -m0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32], pl[kHiLo ? 32 : 1];
#pragma unroll
          for (int b = 4 * half; b < 4 * half + 4; ++b) {
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < kBS; i += 2) {
              float x0, x1;
              f2_split(add2(f2(v[b * kBS + i], v[b * kBS + i + 1]), nm), x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              sum = i == 0 ? f2(x0, x1) : add2(sum, f2(x0, x1));
              const int at = (b - 4 * half) * 8 + i / 2;
              pk[at] = f16x2_of(x0, x1);
              if constexpr (kHiLo) pl[at] = f16x2_rest(pk[at], x0, x1);
            }
            float s0, s1;
            f2_split(sum, s0, s1);
            const float inv = sc[2 * kBlk + b];
            if (inv < 0.f && s0 + s1 > 0.f) record_error(2);  // a table entry outside the pool, and a row that sees it
            l = __fmaf_rn(s0 + s1, fabsf(inv), l);
          }
          __syncwarp();
          tmem_st32(ts + 32 * half, pk);
          if constexpr (kHiLo) tmem_st32(ts + 64 + 32 * half, pl);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&p_full[2 * slot + half]);
        }
      }
      // ---- the end of the segment: O / l, or a record.  The next segment's first
      // product may start before O is read.
      if (asked) hand_q();
      const int last = n - 1;
      float M = Mown, lsum = l;
      if constexpr (!Ly::kPair) {
        named_bar_sync(1, 2 * kWG);  // both warpgroups are through their tiles: S(last) was complete
        M = mref[(last & 1) * kRows + row];
        lrow[wg * kRows + row] = Mown == -INFINITY ? 0.f : l * ex2(Mown - M);
        named_bar_sync(1, 2 * kWG);
        lsum = lrow[row] + lrow[kRows + row];
      }
      pwait(&pv_done[Ly::kPair ? wg : last & 1], Ly::kPair ? last & 1 : (last >> 1) & 1, abort_flag);
      __syncwarp();
      tc_fence_after();
      constexpr int kHalf = Ly::kPair ? D : D / 2;  // columns per warpgroup
      const int col0 = Ly::kPair ? 0 : wg * kHalf;
      const uint32_t to = to0 + col0;
      if (w.first == 0 && w.len == w.cnt) {
        const float iv = lsum > 0.f ? 1.0f / lsum : 0.f;
        // 16-byte units, brought to whole 128-byte lines of a row by transposing
        // among eight lanes (four for 64 bytes): a row per lane costs 32 lines a store
        constexpr int kG = kHiLo || kHalf >= 64 ? 8 : 4;  // lanes, and rows, of a group
        size_t at[kG];
        {
          const size_t mine = valid ? ((size_t)j * p.Hq + hq) * D + col0 : ~(size_t)0;
#pragma unroll
          for (int k = 0; k < kG; ++k) at[k] = __shfl_sync(0xffffffffu, (unsigned long long)mine, (lane & ~(kG - 1)) + k);
        }
        auto put = [&](auto& u, int col) {  // units from column `col` of this warpgroup's part
          constexpr int U = sizeof(u) / 16;
          static_assert(U == kG, "");
          transpose_units<U>(u, lane);
          const int unit = lane % U;
#pragma unroll
          for (int k = 0; k < U; ++k)
            if (at[k] != ~(size_t)0) {
              if constexpr (!kHiLo)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at[k] + col + unit * 8) = u[k];
              else
                *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at[k] + col + unit * 4) = u[k];
            }
        };
        constexpr int kCols = kHiLo || kHalf < 64 ? 32 : 64;  // columns at a time
#pragma unroll 1
        for (int c = 0; c < kHalf; c += kCols) {
          float o[kCols];
#pragma unroll
          for (int i = 0; i < kCols; i += 32) tmem_ld32(to + c + i, *reinterpret_cast<float(*)[32]>(o + i));
          tmem_wait_ld();
          constexpr int U = kHiLo ? 8 : kCols / 8;
          uint4 u[U];
#pragma unroll
          for (int i = 0; i < U; ++i) {
            if constexpr (kHiLo)
              u[i] = make_uint4(__float_as_uint(o[4 * i] * iv), __float_as_uint(o[4 * i + 1] * iv),
                                __float_as_uint(o[4 * i + 2] * iv), __float_as_uint(o[4 * i + 3] * iv));
            else
              u[i] = make_uint4(bf16x2_rn(o[8 * i] * iv, o[8 * i + 1] * iv), bf16x2_rn(o[8 * i + 2] * iv, o[8 * i + 3] * iv),
                                bf16x2_rn(o[8 * i + 4] * iv, o[8 * i + 5] * iv),
                                bf16x2_rn(o[8 * i + 6] * iv, o[8 * i + 7] * iv));
          }
          put(u, c);
        }
      } else {
        // a record: [D / 4][rows] float4, so that neighbouring lanes are neighbours
        float* rec = reinterpret_cast<float*>(ws + pp.w.oRec) +
                     (size_t)(2 * blockIdx.x + (first_seg ? 0 : 1)) * Ly::kRB * (D + 2);
        const int rr = (Ly::kPair ? wg * kRows : 0) + row;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 32) {
          float o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(rec + ((col0 + c + i) / 4 * Ly::kRB + rr) * 4) =
                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
        if (Ly::kPair || wg == 0) {
          rec[Ly::kRB * D + rr] = M;
          rec[Ly::kRB * D + Ly::kRB + rr] = lsum;
        }
      }
      tc_fence_before();
      mbar_arrive(&o_free[Ly::kPair ? wg : 0]);
      first_seg = false;
      w = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Row blocks that span CTAs, merged in CTA order.  The grid runs over the places
// where the list is cut, groups of 32 rows and of 32 columns; a row block's
// first cut has its merge.  lane = row; each of the eight warps takes every eighth
// record, and the eight results are joined in order.
constexpr int kMergeCols = 32;
template <int D>
__global__ void __launch_bounds__(256) block_prefix_merge_kernel(const __grid_constant__ Params pp) {
  constexpr int kQ = kMergeCols / 4, kGroups = D / kMergeCols, kRB = block_rows(D), kParts = kRB / 32;
  __shared__ float s_o[8][32][kMergeCols + 1];
  __shared__ float s_m[8][32], s_l[8][32];
  const BlockDecodeParams& p = pp.a;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cg = blockIdx.x % kGroups, part = blockIdx.x / kGroups % kParts, cut = blockIdx.x / (kParts * kGroups) + 1;
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const int* cuts = reinterpret_cast<const int*>(ws + pp.w.oCuts);
  const int here = cuts[cut], prev = cuts[cut - 1], after = cuts[cut + 1], grid = pp.w.grid, tid = threadIdx.x;
  const int later = cut + 1 + tid < grid ? cuts[cut + 1 + tid] : 0x7fffffff;
  const Head h = reinterpret_cast<const Head*>(ws + pp.w.oHead)[cut];
  if (here >= after || h.first == 0) return;  // an empty range, or no row block is cut here
  const int a = here - h.first, e = a + h.cnt, c0 = cut - 1;  // cuts inside a row block differ
  if (prev > a) return;  // not the first cut of the row block
  const int row = part * 32 + lane, R = p.C * p.G;
  if (h.rb * kRB + part * 32 >= R) return;
  const bool own0 = prev == a;
  int c1 = cut + __syncthreads_count(later < e);  // the last CTA that starts before the row block's end
  for (int c = cut + 257; c < grid; c += 256) c1 += __syncthreads_count(c + tid < grid && cuts[c + tid] < e);
  float4 acc[kQ];
  float M = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kQ; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0 + warp; c <= c1; c += 16) {
    float4 x[2][kQ];
    float m[2], ll[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int cc = c + 8 * k;
      m[k] = -INFINITY;
      if (cc <= c1) {
        // a CTA whose range starts inside the row block has it as its first segment
        const float* rec = reinterpret_cast<const float*>(ws + pp.w.oRec) + (size_t)(2 * cc + (cc > c0 || own0 ? 0 : 1)) * kRB * (D + 2);
#pragma unroll
        for (int i = 0; i < kQ; ++i) x[k][i] = *reinterpret_cast<const float4*>(rec + ((cg * kQ + i) * kRB + row) * 4);
        m[k] = rec[kRB * D + row];
        ll[k] = rec[kRB * D + kRB + row];
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (m[k] == -INFINITY) continue;
      const float nm = fmaxf(M, m[k]);
      const float f = ex2(M - nm), g = ex2(m[k] - nm);
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        acc[i].x = acc[i].x * f + x[k][i].x * g;
        acc[i].y = acc[i].y * f + x[k][i].y * g;
        acc[i].z = acc[i].z * f + x[k][i].z * g;
        acc[i].w = acc[i].w * f + x[k][i].w * g;
      }
      l = l * f + ll[k] * g;
      M = nm;
    }
  }
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    s_o[warp][lane][4 * i] = acc[i].x;
    s_o[warp][lane][4 * i + 1] = acc[i].y;
    s_o[warp][lane][4 * i + 2] = acc[i].z;
    s_o[warp][lane][4 * i + 3] = acc[i].w;
  }
  s_m[warp][lane] = M;
  s_l[warp][lane] = l;
  __syncthreads();
  // lane = column now; four rows per warp
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = warp * 4 + i, r = h.rb * kRB + part * 32 + rr;
    if (r >= R) break;
    float C = -INFINITY, den = 0.f, o = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) C = fmaxf(C, s_m[k][rr]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s_m[k][rr] == -INFINITY) continue;
      const float f = ex2(s_m[k][rr] - C);
      den = __fmaf_rn(s_l[k][rr], f, den);
      o = __fmaf_rn(s_o[k][rr][lane], f, o);
    }
    const float v = den > 0.f ? o / den : 0.f;
    const int j = p.divG.div(r);
    store_out1(p.out, p.out_bf16, ((size_t)j * p.Hq + h.kvh * p.G + r - j * p.G) * D + cg * kMergeCols + lane, v);
  }
}

// The same for row blocks of a few records each: a warp has 32 rows and 32 columns
// of its own, and goes through the records two at a time.
template <int D>
__global__ void __launch_bounds__(256) block_prefix_join_kernel(const __grid_constant__ Params pp) {
  constexpr int kQ = kMergeCols / 4, kGroups = D / kMergeCols, kRB = block_rows(D), kSets = kRB / 32 * kGroups / 8;
  const BlockDecodeParams& p = pp.a;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int cut = blockIdx.x / kSets + 1, set = blockIdx.x % kSets * 8 + warp;
  const int cg = set % kGroups, part = set / kGroups;
  uint8_t* ws = static_cast<uint8_t*>(p.ws);
  const int* cuts = reinterpret_cast<const int*>(ws + pp.w.oCuts);
  const int here = cuts[cut], prev = cuts[cut - 1], after = cuts[cut + 1], grid = pp.w.grid;
  const int later = cut + 1 + tid < grid ? cuts[cut + 1 + tid] : 0x7fffffff;
  const Head h = reinterpret_cast<const Head*>(ws + pp.w.oHead)[cut];
  if (here >= after || h.first == 0) return;  // an empty range, or no row block is cut here
  const int a = here - h.first, e = a + h.cnt, c0 = cut - 1;  // cuts inside a row block differ
  if (prev > a) return;  // not the first cut of the row block
  const bool own0 = prev == a;
  int c1 = cut + __syncthreads_count(later < e);  // the last CTA that starts before the row block's end
  for (int c = cut + 257; c < grid; c += 256) c1 += __syncthreads_count(c + tid < grid && cuts[c + tid] < e);
  const int row = part * 32 + lane, r = h.rb * kRB + row, R = p.C * p.G;
  if (r - lane >= R) return;
  float4 acc[kQ];
  float M = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < kQ; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= c1; c += 2) {
    float4 x[2][kQ];
    float m[2], ll[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int cc = c + k;
      m[k] = -INFINITY;
      if (cc <= c1) {
        // a CTA whose range starts inside the row block has it as its first segment
        const float* rec = reinterpret_cast<const float*>(ws + pp.w.oRec) + (size_t)(2 * cc + (cc > c0 || own0 ? 0 : 1)) * kRB * (D + 2);
#pragma unroll
        for (int i = 0; i < kQ; ++i) x[k][i] = *reinterpret_cast<const float4*>(rec + ((cg * kQ + i) * kRB + row) * 4);
        m[k] = rec[kRB * D + row];
        ll[k] = rec[kRB * D + kRB + row];
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (m[k] == -INFINITY) continue;
      const float nm = fmaxf(M, m[k]);
      const float f = ex2(M - nm), g = ex2(m[k] - nm);
#pragma unroll
      for (int i = 0; i < kQ; ++i) {
        acc[i].x = acc[i].x * f + x[k][i].x * g;
        acc[i].y = acc[i].y * f + x[k][i].y * g;
        acc[i].z = acc[i].z * f + x[k][i].z * g;
        acc[i].w = acc[i].w * f + x[k][i].w * g;
      }
      l = l * f + ll[k] * g;
      M = nm;
    }
  }
  const float iv = l > 0.f ? 1.0f / l : 0.f;
  // 16-byte units, exchanged among the lanes of a group so that a row's line is whole
  const int j = p.divG.div(r);
  const size_t mine = r < R ? ((size_t)j * p.Hq + h.kvh * p.G + r - j * p.G) * D + cg * kMergeCols : ~(size_t)0;
  auto put = [&](auto& u) {
    constexpr int U = sizeof(u) / 16;
    transpose_units<U>(u, lane);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const size_t at = __shfl_sync(0xffffffffu, (unsigned long long)mine, (lane & ~(U - 1)) + k);
      if (at == ~(size_t)0) continue;
      if constexpr (U == 4)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at + lane % U * 8) = u[k];
      else
        *reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at + lane % U * 4) = u[k];
    }
  };
  if (p.out_bf16) {
    uint4 u[kQ / 2];
#pragma unroll
    for (int i = 0; i < kQ / 2; ++i)
      u[i] = make_uint4(bf16x2_rn(acc[2 * i].x * iv, acc[2 * i].y * iv), bf16x2_rn(acc[2 * i].z * iv, acc[2 * i].w * iv),
                        bf16x2_rn(acc[2 * i + 1].x * iv, acc[2 * i + 1].y * iv),
                        bf16x2_rn(acc[2 * i + 1].z * iv, acc[2 * i + 1].w * iv));
    put(u);
  } else {
    uint4 u[kQ];
#pragma unroll
    for (int i = 0; i < kQ; ++i)
      u[i] = make_uint4(__float_as_uint(acc[i].x * iv), __float_as_uint(acc[i].y * iv), __float_as_uint(acc[i].z * iv),
                        __float_as_uint(acc[i].w * iv));
    put(u);
  }
}

template <int D, bool kCap, bool kSlope, bool kHiLo>
cudaError_t launch(const Params& pp, cudaStream_t stream) {
  auto* kernel = block_prefix_kernel<D, kCap, kSlope, kHiLo>;
  // the shared-memory opt-in, once per device (graph captures then make no attribute call)
  int dev = 0;
  cudaGetDevice(&dev);
  static bool opted[64] = {false};
  if (dev < 0 || dev >= 64 || !opted[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kTotal);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) opted[dev] = true;
  }
  cudaError_t e = launch_pdl(block_tiles_kernel<D>, dim3(pp.w.ntiles, pp.a.Hkv, 2), dim3(256), 0, stream, pp);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3(pp.w.grid), dim3(kThreads), Lay<D>::kTotal, stream, pp);
  if (e != cudaSuccess || pp.w.grid == 1) return e;
  const int sets = (block_rows(D) / 32) * (D / kMergeCols);
  // Up to some eight records a row block (on average; masks may leave one with more):
  // a warp per 32 x 32 of it.  Row blocks 384 (24/4/256, 2048 rows over 16384 keys)
  // 545 -> 517 us, 19 (16/1/128, 300 over 8192) 46 -> 42; 12 (24/4/256, 64 over 8192)
  // 46 -> 47.5.
  if ((int64_t)pp.w.nrb * pp.a.Hkv * 8 >= pp.w.grid)
    return launch_pdl(block_prefix_join_kernel<D>, dim3((pp.w.grid - 1) * (sets / 8)), dim3(256), 0, stream, pp);
  return launch_pdl(block_prefix_merge_kernel<D>, dim3((pp.w.grid - 1) * sets), dim3(256), 0, stream, pp);
}

template <int D, bool kHiLo>
cudaError_t launch_w(const Params& pp, cudaStream_t stream) {
  const bool cap = pp.a.cap_log2 > 0.f, slope = pp.a.slopes != nullptr;
  if (cap) return slope ? launch<D, true, true, kHiLo>(pp, stream) : launch<D, true, false, kHiLo>(pp, stream);
  return slope ? launch<D, false, true, kHiLo>(pp, stream) : launch<D, false, false, kHiLo>(pp, stream);
}

template <int D>
cudaError_t launch_any(const Params& pp, cudaStream_t stream) {
  return pp.a.out_bf16 ? launch_w<D, false>(pp, stream) : launch_w<D, true>(pp, stream);
}

}  // namespace bp
}  // namespace i8kv
