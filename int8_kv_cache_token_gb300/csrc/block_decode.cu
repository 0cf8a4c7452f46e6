// block_decode.cu -- decode attention over the block-scaled INT8 KV cache, with
// an optional tanh cap, distance bias, sliding window and first visible key.
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
// order.
#include "common.cuh"
#include "kernels.h"

namespace i8kv {
I8KV_DEFINE_ERROR_ACCESSOR(read_error_block_decode)

namespace {

constexpr int kBS = 16;
constexpr int kHeads = 8;        // query rows per pass: the MMA's N
constexpr float kLazy = 8.0f;    // log2 units by which a score may pass M

template <int D>
struct Geo {
  static constexpr int kWarps = D == 256 ? 8 : 16;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kPage = D * kBS;
  static constexpr int kStages = D == 256 ? 3 : D == 128 ? 3 : 6;  // pages in flight per warp
  static constexpr int kStage = 2 * kPage;
  static constexpr int kRow = D + 4;                  // floats per head of a merge buffer (conflict-free)
  static constexpr int kBufs = 4;                     // merge buffers
  static constexpr int oRing = 0;
  static constexpr int oMerge = oRing + kWarps * kStages * kStage;
  static constexpr int oScale = oMerge + kBufs * kHeads * kRow * 4;  // float2 (sK, sV) per stage
  static constexpr int oBar = oScale + kWarps * kStages * 8;
  static constexpr int oStat = oBar + kWarps * kStages * 8;          // M, l [kWarps][8] each
  static constexpr int oScan = oStat + 2 * kWarps * kHeads * 4;
  static constexpr int kTotal = oScan + 64 * 8;
  static_assert(kTotal <= 232448, "shared memory");
};

// The workspace: a header per CTA (where its range starts), then two partial
// records per CTA (its first and its last segment), each o [8][D], M [8], l [8].
struct Head {
  int b, hh;         // sequence and head pass; b = -1: an empty range
  int first;         // visible blocks of the pair before the range
  int nb;            // visible blocks of the pair
  long long total;   // blocks of the flattened list
  long long unused;
};
static_assert(sizeof(Head) == 32, "16-byte aligned records");
__host__ __device__ constexpr int rec_floats(int D) { return kHeads * D + 2 * kHeads; }
__device__ __forceinline__ float* record(const BlockDecodeParams& p, int slot, int D) {
  return reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + (size_t)p.grid * sizeof(Head)) + (size_t)slot * rec_floats(D);
}

// One entry of the work list: a sequence (decode), or eight (token, head) rows of
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
  if (p.key_end != nullptr) hi = min(p.key_end[j], p.H + p.C);
}

template <bool kChunk>
__device__ __forceinline__ Seq seq_of(const BlockDecodeParams& p, int b) {
  Seq s;
  if constexpr (kChunk) {
    s.lo = s.hi_in = 0x7fffffff;
    s.hi = s.lo_in = 0;
    const int j1 = min(p.C - 1, (b * kHeads + kHeads - 1) / p.G);
    for (int j = b * kHeads / p.G; j <= j1; ++j) {
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

// Row c (0 .. 7) of head pass hh of entry b: its token (the row of q and out
// and of the masks) and query head; false where there is none.
template <bool kChunk>
__device__ __forceinline__ bool row_of(const BlockDecodeParams& p, int b, int hh, int c, int& tok, int& head) {
  if constexpr (kChunk) {
    const int r = b * kHeads + c;
    tok = r / p.G;
    head = hh * p.G + r % p.G;
    return r < p.C * p.G;
  } else {
    const int in = (hh % p.HG) * kHeads + c;
    tok = b;
    head = hh / p.HG * p.G + in;
    return in < p.G;
  }
}

// A warp's walk over the blocks of its CTA's range [u, u1) of the flattened
// list (sequence, head pass, block).
struct Walk {
  int b, hh;          // current sequence and head pass
  long long left;     // blocks of the range from here on, this segment's included
  Seq s;
  int first, len;     // this segment: visible blocks [first, first + len) of the sequence
};

__device__ __forceinline__ void walk_segment(Walk& w) {
  w.len = (int)min((long long)(w.s.nb - w.first), w.left);
}
// To the next segment; false at the end of the range.
template <bool kChunk>
__device__ __forceinline__ bool walk_next(const BlockDecodeParams& p, Walk& w) {
  w.left -= w.len;
  if (w.left <= 0) return false;
  w.first = 0;
  if (++w.hh == p.HH) {
    w.hh = 0;
    do {
      if (++w.b >= p.B) return false;  // only if the lengths changed under the kernel
      w.s = seq_of<kChunk>(p, w.b);
    } while (w.s.nb == 0);
  }
  walk_segment(w);
  return true;
}

// Sum over the CTA's threads, and the sum over the threads before this one.
template <int NW>
__device__ __forceinline__ long long cta_scan(long long v, long long& before, long long* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  long long base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < warp) base += buf[i];
    total += buf[i];
  }
  before = base + x - v;
  return total;
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
// kChunk: the work list holds the rows of one sequence's chunk.
template <int D, bool kChunk, bool kCap, bool kHiLo>
__global__ void __launch_bounds__(Geo<D>::kThreads, 1) block_decode_kernel(BlockDecodeParams p) {
  using Gm = Geo<D>;
  constexpr int NW = Gm::kWarps, NS = Gm::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint8_t* ring = smem + Gm::oRing + (size_t)warp * NS * Gm::kStage;
  float* merge = reinterpret_cast<float*>(smem + Gm::oMerge);
  float2* scl = reinterpret_cast<float2*>(smem + Gm::oScale) + warp * NS;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Gm::oBar) + warp * NS;
  float* statM = reinterpret_cast<float*>(smem + Gm::oStat);
  float* statL = statM + NW * kHeads;
  long long* scan = reinterpret_cast<long long*>(smem + Gm::oScan);

  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&bar[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's range of the flattened list, and where it starts ----
  long long total = 0, mine;
  for (int b0 = 0; b0 < p.B; b0 += Gm::kThreads) {
    const int b = b0 + tid;
    const int nb = b < p.B ? seq_of<kChunk>(p, b).nb : 0;
    if (!kChunk && b < p.B && blockIdx.x == 0 && p.seq_lens[b] > p.max_blocks * kBS) record_error(2);
    total += cta_scan<NW>(nb, mine, scan);
  }
  total *= p.HH;
  const long long u0 = total * blockIdx.x / gridDim.x, u1 = total * (blockIdx.x + 1) / gridDim.x;
  // entries without a visible key: zero rows
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (seq_of<kChunk>(p, b).nb == 0)
      for (int i = tid; i < p.HH * kHeads * (D / 4); i += Gm::kThreads) {
        const int c4 = (i % (D / 4)) * 4, c = i / (D / 4);
        int tok, hd;
        if (row_of<kChunk>(p, b, c / kHeads, c % kHeads, tok, hd))
          store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + c4, make_float4(0.f, 0.f, 0.f, 0.f));
      }
  Head* head = static_cast<Head*>(p.ws) + blockIdx.x;
  if (u0 >= u1) {
    if (tid == 0) head->b = -1;
    return;
  }
  int* start = reinterpret_cast<int*>(scan + 32);  // sequence, head pass, block
  if (tid < 3) start[tid] = 0;
  long long run = 0;
  for (int b0 = 0; b0 < p.B; b0 += Gm::kThreads) {
    const int b = b0 + tid;
    const int nb = b < p.B ? seq_of<kChunk>(p, b).nb : 0;
    const long long sum = cta_scan<NW>(nb, mine, scan);
    const long long s0 = (run + mine) * p.HH;
    if (u0 >= s0 && u0 < s0 + (long long)nb * p.HH) {
      start[0] = b;
      start[1] = (int)((u0 - s0) / nb);
      start[2] = (int)((u0 - s0) % nb);
    }
    run += sum;
  }
  __syncthreads();
  Walk w;
  w.b = start[0];
  w.hh = start[1];
  w.first = start[2];
  w.left = u1 - u0;
  w.s = seq_of<kChunk>(p, w.b);
  walk_segment(w);
  if (tid == 0) *head = Head{w.b, w.hh, w.first, w.s.nb, total, 0};

  // ---- the page copies: a walk of their own, NS blocks ahead of the consumer ----
  Walk c = w;
  int c_i = warp;        // next block of the segment for this warp
  int c_n = 0;           // blocks asked for so far (slot c_n % NS)
  bool c_more = true;    // false: the range is done, or a wait ran out of time
  int table = 0, table_at = -1;  // lane i: the table entry of the warp's block table_at + i of the segment
  auto issue = [&]() {
    if (!c_more) return;
    while (c_i >= c.len) {
      if (!walk_next<kChunk>(p, c)) {
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
    const int kvh = kChunk ? c.hh : c.hh / p.HG;
    const int slot = c_n % NS;
    const size_t ph = (size_t)phys * p.Hkv + kvh;
    if (lane == 0) mbar_expect_tx(&bar[slot], Gm::kStage);
    __syncwarp();
    if (lane == 0) {
      bulk_g2s(ring + slot * Gm::kStage, p.k_cache + ph * Gm::kPage, Gm::kPage, &bar[slot]);
      bulk_g2s(ring + slot * Gm::kStage + Gm::kPage, p.v_cache + ph * Gm::kPage, Gm::kPage, &bar[slot]);
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
    // the rows of this lane: row g as a row of q, rows 2 t4 and 2 t4 + 1 as columns
    // of the scores and the output
    int q_tok, q_head;
    const bool q_row = row_of<kChunk>(p, w.b, w.hh, g, q_tok, q_head);
    int lo0 = w.s.lo, hi0 = w.s.hi, lo1 = w.s.lo, hi1 = w.s.hi, pos0 = w.s.hi - 1, pos1 = w.s.hi - 1;
    float sl0 = 0.f, sl1 = 0.f;
    {
      int tok, hd;
      if (row_of<kChunk>(p, w.b, w.hh, 2 * t4, tok, hd)) {
        if (p.slopes != nullptr) sl0 = -__ldg(p.slopes + hd) * kLog2e;
        if constexpr (kChunk) {
          chunk_interval(p, tok, lo0, hi0);
          pos0 = p.H + tok;
        }
      }
      if (row_of<kChunk>(p, w.b, w.hh, 2 * t4 + 1, tok, hd)) {
        if (p.slopes != nullptr) sl1 = -__ldg(p.slopes + hd) * kLog2e;
        if constexpr (kChunk) {
          chunk_interval(p, tok, lo1, hi1);
          pos1 = p.H + tok;
        }
      }
    }
    // q of row g as the B operand: dims 16 c + 4 t4 .. + 3 of chunk c,
    // scaled by a power of two that brings the row's maximum near 2^14
    uint32_t qf[D / 16][2];
    float qs;
    {
      uint2 raw[D / 16];
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        raw[i] = make_uint2(0, 0);
        if (q_row)
          raw[i] = __ldg(reinterpret_cast<const uint2*>(p.q + (int64_t)q_tok * p.q_stride + (size_t)q_head * D + 16 * i + 4 * t4));
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        am = fmaxf(am, fmaxf(fabsf(__uint_as_float(raw[i].x << 16)), fabsf(__uint_as_float(raw[i].x & 0xffff0000u))));
        am = fmaxf(am, fmaxf(fabsf(__uint_as_float(raw[i].y << 16)), fabsf(__uint_as_float(raw[i].y & 0xffff0000u))));
      }
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int ex = max(-100, (int)(__float_as_uint(am) >> 23) - 127);  // -100: zero rows and values below 2^-100
      const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
      qs = __uint_as_float((uint32_t)(ex - 14 + 127) << 23) * p.score_mul;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        qf[i][0] = f16x2_of(__uint_as_float(raw[i].x << 16) * up, __uint_as_float(raw[i].x & 0xffff0000u) * up);
        qf[i][1] = f16x2_of(__uint_as_float(raw[i].y << 16) * up, __uint_as_float(raw[i].y & 0xffff0000u) * up);
      }
    }
    const float qs0 = __shfl_sync(0xffffffffu, qs, 8 * t4), qs1 = __shfl_sync(0xffffffffu, qs, 8 * t4 + 4);
    float o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float M0 = -INFINITY, M1 = -INFINITY, l0 = 0.f, l1 = 0.f;

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
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[0][j] = s[1][j] = 0.f;
#pragma unroll
      for (int ch = 0; ch < D / 16; ch += 2) {
        uint32_t a[4], lo[4], hi[4];
        ldmatrix_x4(a, kp + ch * (kBS * 16) + k_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) s8x4_to_f16(a[j], lo[j], hi[j]);
        mma_f16_16816(s[0], lo[0], lo[1], hi[0], hi[1], qf[ch][0], qf[ch][1]);
        mma_f16_16816(s[1], lo[2], lo[3], hi[2], hi[3], qf[ch + 1][0], qf[ch + 1][1]);
      }
      // u = score log2 e + log2 sV.  A block of zero V codes (sV = 0) gets the
      // floor 2^-100: its codes add nothing, its weights still count in l.
      const float svf = fmaxf(sv, kTinyDivisor);
      const float lv = kHiLo ? log2f(svf) : __log2f(svf), inv = __frcp_rn(svf);
      const float c0 = qs0 * sk, c1 = qs1 * sk;
      float u[4] = {s[0][0] + s[1][0], s[0][1] + s[1][1], s[0][2] + s[1][2], s[0][3] + s[1][3]};
      const int key0 = (w.s.fb + w.first + i) * kBS;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] *= (j & 1) ? c1 : c0;
      if constexpr (kCap) {
        // u = score / cap here; cap log2 e tanh u, by the polynomial in u^2 for |u| <= 1
        if (__any_sync(0xffffffffu, !(fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3]))) <= 1.f))) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            u[j] = kHiLo ? __fmaf_rn(p.cap_log2, tanhf(u[j]), lv)
                         : __fmaf_rn(-2.f * p.cap_log2, rcp_approx(ex2(u[j] * (2.f * kLog2e)) + 1.f), p.cap_log2 + lv);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float y = u[j] * u[j];
            float a = p.cap_poly[kCapDeg];
#pragma unroll
            for (int d = kCapDeg - 1; d >= 0; --d) a = __fmaf_rn(a, y, p.cap_poly[d]);
            u[j] = __fmaf_rn(a, u[j], lv);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] += lv;
      }
      if (p.slopes != nullptr) {
        u[0] = __fmaf_rn(sl0, (float)abs(key0 + tok0 - pos0), u[0]);
        u[1] = __fmaf_rn(sl1, (float)abs(key0 + tok0 - pos1), u[1]);
        u[2] = __fmaf_rn(sl0, (float)abs(key0 + tok1 - pos0), u[2]);
        u[3] = __fmaf_rn(sl1, (float)abs(key0 + tok1 - pos1), u[3]);
      }
      if (key0 < w.s.lo_in || key0 + kBS > w.s.hi_in) {  // a block with hidden tokens
        if (key0 + tok0 < lo0 || key0 + tok0 >= hi0) u[0] = -INFINITY;
        if (key0 + tok0 < lo1 || key0 + tok0 >= hi1) u[1] = -INFINITY;
        if (key0 + tok1 < lo0 || key0 + tok1 >= hi0) u[2] = -INFINITY;
        if (key0 + tok1 < lo1 || key0 + tok1 >= hi1) u[3] = -INFINITY;
      }
      // M moves for all the lanes of a head together
      if (__any_sync(0xffffffffu, fmaxf(u[0], u[2]) > M0 + kLazy || fmaxf(u[1], u[3]) > M1 + kLazy)) {
        float m0 = fmaxf(M0, fmaxf(u[0], u[2])), m1 = fmaxf(M1, fmaxf(u[1], u[3]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
          m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
        }
        const float a0 = M0 == -INFINITY ? 0.f : ex2(M0 - m0), a1 = M1 == -INFINITY ? 0.f : ex2(M1 - m1);
        M0 = m0;
        M1 = m1;
        l0 *= a0;
        l1 *= a1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          o[k][0] *= a0;
          o[k][1] *= a1;
          o[k][2] *= a0;
          o[k][3] *= a1;
        }
      }
      // a row that has seen no key yet: M = -inf, weights 0
      const float n0 = kChunk && M0 == -INFINITY ? 0.f : M0, n1 = kChunk && M1 == -INFINITY ? 0.f : M1;
      const float w0 = ex2(u[0] - n0), w1 = ex2(u[1] - n1), w2 = ex2(u[2] - n0), w3 = ex2(u[3] - n1);
      l0 = __fmaf_rn(w0 + w2, inv, l0);
      l1 = __fmaf_rn(w1 + w3, inv, l1);
      // [token][head] -> the B operand [head][token pairs]; for t4 >= 2 the upper
      // half holds tokens 4 t4 + 2, + 3
      const uint32_t p0 = f16x2_of(w0, w1), p1 = f16x2_of(w2, w3);
      const uint32_t x0 = movmatrix_trans(p0), x1 = movmatrix_trans(p1);
      const uint32_t b0 = t4 < 2 ? x0 : x1, b1 = t4 < 2 ? x1 : x0;
      uint32_t e0 = 0, e1 = 0;
      if constexpr (kHiLo) {
        const uint32_t y0 = movmatrix_trans(f16x2_rest(p0, w0, w1)), y1 = movmatrix_trans(f16x2_rest(p1, w2, w3));
        e0 = t4 < 2 ? y0 : y1;
        e1 = t4 < 2 ? y1 : y0;
      }
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) {  // 32 dims: two row tiles of the MMA
        uint32_t a[4], lo[4], hi[4];
        ldmatrix_x4(a, vp + dt * (32 * 16) + v_off);
#pragma unroll
        for (int j = 0; j < 4; ++j) s8x4_to_f16(a[j], lo[j], hi[j]);
        mma_f16_16816(o[2 * dt], lo[0], lo[1], hi[0], hi[1], b0, b1);
        mma_f16_16816(o[2 * dt + 1], lo[2], lo[3], hi[2], hi[3], b0, b1);
        if constexpr (kHiLo) {
          mma_f16_16816(o[2 * dt], lo[0], lo[1], hi[0], hi[1], e0, e1);
          mma_f16_16816(o[2 * dt + 1], lo[2], lo[3], hi[2], hi[3], e0, e1);
        }
      }
      __syncwarp();  // every lane is done with the slot
      issue();
    }

    // ---- the warps' (o, M, l) of this segment joined, in a fixed order ----
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (g == 0) {
      statM[warp * kHeads + 2 * t4] = M0;
      statM[warp * kHeads + 2 * t4 + 1] = M1;
      statL[warp * kHeads + 2 * t4] = l0;
      statL[warp * kHeads + 2 * t4 + 1] = l1;
    }
    __syncthreads();
    float C0 = -INFINITY, C1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      C0 = fmaxf(C0, statM[i * kHeads + 2 * t4]);
      C1 = fmaxf(C1, statM[i * kHeads + 2 * t4 + 1]);
    }
    const float f0 = M0 == -INFINITY ? 0.f : ex2(M0 - C0), f1 = M1 == -INFINITY ? 0.f : ex2(M1 - C1);
    float* buf = merge + (warp % Gm::kBufs) * (kHeads * Gm::kRow);
#pragma unroll 1
    for (int r = NW / Gm::kBufs - 1; r >= 0; --r) {  // four warps at a time, the last ones first
      if (warp / Gm::kBufs == r) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& x = buf[(2 * t4 + (j & 1)) * Gm::kRow + 16 * k + g + (j >> 1) * 8];
            x = __fmaf_rn(o[k][j], (j & 1) ? f1 : f0, r == NW / Gm::kBufs - 1 ? 0.f : x);
          }
      }
      __syncthreads();
    }
    const bool whole = w.first == 0 && w.len == w.s.nb;
    float* rec = record(p, 2 * blockIdx.x + (first_seg ? 0 : 1), D);
    for (int i = tid; i < kHeads * D / 4; i += Gm::kThreads) {
      const int h = i / (D / 4), c4 = (i % (D / 4)) * 4;
      int tok, hd;
      if (!row_of<kChunk>(p, w.b, w.hh, h, tok, hd)) continue;
      float4 acc = *reinterpret_cast<const float4*>(merge + h * Gm::kRow + c4);
#pragma unroll
      for (int k = 1; k < Gm::kBufs; ++k) {
        const float4 x = *reinterpret_cast<const float4*>(merge + (k * kHeads + h) * Gm::kRow + c4);
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      float C = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) C = fmaxf(C, statM[k * kHeads + h]);
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float m = statM[k * kHeads + h];
        if (m != -INFINITY) l = __fmaf_rn(statL[k * kHeads + h], ex2(m - C), l);
      }
      if (whole) {
        const float iv = l > 0.f ? 1.0f / l : 0.f;  // a row without a visible key is zero
        store_out4(p.out, p.out_bf16, ((size_t)tok * p.Hq + hd) * D + c4,
                   make_float4(acc.x * iv, acc.y * iv, acc.z * iv, acc.w * iv));
      } else {
        *reinterpret_cast<float4*>(rec + h * D + c4) = acc;
        if (c4 == 0) {
          rec[kHeads * D + h] = C;
          rec[kHeads * D + kHeads + h] = l;
        }
      }
    }
    first_seg = false;
    if (!walk_next<kChunk>(p, w)) break;
    __syncthreads();  // the merge buffers are free again
  }
  // after a time-out: the copies still under way get one more (bounded) wait
  if (__any_sync(0xffffffffu, dead))
    for (int k = max(0, c_n - NS); k < c_n; ++k) mbar_wait(&bar[k % NS], (k / NS) & 1);
}

// The records of the pairs that span CTAs, merged in CTA order.  A pair is cut
// only where a CTA's range starts, so the grid runs over those places (c0 + 1 ..)
// and heads; the first cut inside a pair has its merge.  D / 4 columns of threads
// in kParts parts, each part every kParts-th record.
constexpr int kMergeThreads = 256;

template <int D, bool kChunk>
__global__ void __launch_bounds__(kMergeThreads) block_decode_merge_kernel(BlockDecodeParams p, int heads) {
  constexpr int kCols = D / 4, kParts = kMergeThreads / kCols;
  __shared__ float4 s_o[kParts][kCols];
  __shared__ float s_ml[kParts][2];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const int h = blockIdx.x % heads, cut = blockIdx.x / heads + 1;
  const Head hd = static_cast<const Head*>(p.ws)[cut];
  if (hd.b < 0 || hd.first == 0) return;  // an empty range, or no pair is cut here
  int tok, qh;
  if (!row_of<kChunk>(p, hd.b, hd.hh, h, tok, qh)) return;
  const size_t orow = ((size_t)tok * p.Hq + qh) * D;
  const long long total = hd.total, grid = p.grid;
  auto begin_of = [&](long long c) { return total * c / grid; };
  auto cta_of = [&](long long u) { return (int)(((u + 1) * grid - 1) / total); };
  // the pair's blocks [a, e) of the flattened list lie in the ranges of CTAs c0 .. c1
  const long long a = begin_of(cut) - hd.first, e = a + hd.nb;
  const int c0 = cta_of(a), c1 = cta_of(e - 1);
  if (cut != cta_of(begin_of(c0 + 1))) return;  // not the first cut of the pair
  const int col = tid % kCols, part = tid / kCols;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0 + part; c <= c1; c += kParts) {
    if (begin_of(c) == begin_of(c + 1)) continue;  // an empty range (fewer blocks than CTAs)
    // a CTA whose range starts inside the pair has it as its first segment
    const float* rec = record(p, 2 * c + (begin_of(c) >= a ? 0 : 1), D);
    const float4 x = *reinterpret_cast<const float4*>(rec + h * D + 4 * col);
    const float m = rec[kHeads * D + h], ll = rec[kHeads * D + kHeads + h];
    const float nm = fmaxf(M, m);
    if (nm != -INFINITY) {
      const float f = ex2(M - nm), k = ex2(m - nm);  // 2^-inf = 0
      acc.x = acc.x * f + x.x * k;
      acc.y = acc.y * f + x.y * k;
      acc.z = acc.z * f + x.z * k;
      acc.w = acc.w * f + x.w * k;
      l = l * f + ll * k;
      M = nm;
    }
  }
  s_o[part][col] = acc;
  if (col == 0) {
    s_ml[part][0] = M;
    s_ml[part][1] = l;
  }
  __syncthreads();
  if (part == 0) {
    float C = -INFINITY;
#pragma unroll
    for (int k = 0; k < kParts; ++k) C = fmaxf(C, s_ml[k][0]);
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      if (s_ml[k][0] == -INFINITY) continue;
      const float f = ex2(s_ml[k][0] - C);
      const float4 x = s_o[k][col];
      r.x += x.x * f;
      r.y += x.y * f;
      r.z += x.z * f;
      r.w += x.w * f;
      den += s_ml[k][1] * f;
    }
    const float iv = den > 0.f ? 1.0f / den : 0.f;
    store_out4(p.out, p.out_bf16, orow + 4 * col, make_float4(r.x * iv, r.y * iv, r.z * iv, r.w * iv));
  }
}

template <int D, bool kChunk, bool kCap, bool kHiLo>
cudaError_t launch_d(const BlockDecodeParams& p, cudaStream_t stream) {
  auto* kernel = block_decode_kernel<D, kChunk, kCap, kHiLo>;
  // the shared-memory opt-in, once per device (graph captures then make no attribute call)
  int dev = 0;
  cudaGetDevice(&dev);
  static bool opted[64] = {false};
  if (dev < 0 || dev >= 64 || !opted[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::kTotal);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) opted[dev] = true;
  }
  const cudaError_t e = launch_pdl(kernel, dim3(p.grid), dim3(Geo<D>::kThreads), Geo<D>::kTotal, stream, p);
  if (e != cudaSuccess) return e;
  if (p.grid == 1) return cudaSuccess;
  const int heads = !kChunk && p.G < kHeads ? p.G : kHeads;
  return launch_pdl(block_decode_merge_kernel<D, kChunk>, dim3((p.grid - 1) * heads), dim3(kMergeThreads), 0, stream, p,
                    heads);
}

template <int D, bool kChunk>
cudaError_t launch_v(const BlockDecodeParams& p, cudaStream_t stream) {
  const bool cap = p.cap_log2 > 0.f;
  if (p.out_bf16) return cap ? launch_d<D, kChunk, true, false>(p, stream) : launch_d<D, kChunk, false, false>(p, stream);
  return cap ? launch_d<D, kChunk, true, true>(p, stream) : launch_d<D, kChunk, false, true>(p, stream);
}

int device_sms() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 1;
  return n;
}

}  // namespace

// CTAs of the attention kernel: one per SM, or one per block where there are fewer.
int block_decode_grid(int entries, int HH, int max_blocks) {
  const long long most = (long long)entries * HH * max_blocks;
  const int sms = device_sms();
  return most < sms ? (int)(most > 0 ? most : 1) : sms;
}

size_t block_decode_workspace_bytes(int D, int grid) {
  return (size_t)grid * (sizeof(Head) + 2 * rec_floats(D) * sizeof(float));
}

cudaError_t launch_block_decode(const BlockDecodeParams& p, cudaStream_t stream) {
  if (p.D == 256) return launch_v<256, false>(p, stream);
  if (p.D == 128) return launch_v<128, false>(p, stream);
  return launch_v<64, false>(p, stream);
}

cudaError_t launch_block_chunk_rows(const BlockDecodeParams& p, cudaStream_t stream) {
  if (p.D == 256) return launch_v<256, true>(p, stream);
  if (p.D == 128) return launch_v<128, true>(p, stream);
  return launch_v<64, true>(p, stream);
}

}  // namespace i8kv
