// block_cache.cu -- the block-scaled INT8 KV cache: writing tokens into it and
// reading them back.
//
// The pages are the INT8 cache's (K [NB, Hkv, D/16, 16, 16], V [NB, Hkv, D,
// 16]), but K and V have one fp32 scale per (16-token block, KV head):
//   s  = max(s_old, RN(max |x| / 127))   over the block's new tokens; s_old counts
//        only when tokens stand before the first new one in the block
//   new token:    code = RNE(RN(x / s))
//   older token:  code = RNE(RN(code * RN(s_old / s)))   when s != s_old
// Every step is one correctly rounded fp32 operation, so the bytes are
// reproducible (RNE = round half to even).
//
// A call takes a ragged batch: sequence b brings the tokens cu[b] .. cu[b+1]-1,
// which are its last positions.  One CTA owns one (touched block, KV head):
// nothing is shared between CTAs, so growing a scale needs no atomics and no
// second pass.  D threads: the lower half takes the K page, the upper half the
// V page, 64 bytes of bf16 per thread.  All loads (new rows, old codes, old
// scale) are issued before the first of them is used.
//
// Reading back 62 K tokens (8 heads of 128, bf16) takes 64 us, 6.4 TB/s, 0.95 of
// the measured copy rate.  A chunk of 5 K tokens written and read back takes 17 us
// (68 MB, 10 us at the copy rate): the lengths and the table are two round trips
// before a CTA's data.  One token per sequence: 2.7 us, the launch and three
// round trips.
#include "common.cuh"
#include "kernels.h"

namespace i8kv {
I8KV_DEFINE_ERROR_ACCESSOR(read_error_block_cache)

namespace {

constexpr int kBS = 16;

// One block that a ragged call touches.
struct Span {
  int phys;  // its place in the pool
  int f, e;  // the call's tokens are offsets [f, e) of the block
  int tok0;  // offset o is the call's token tok0 + o
};

// Work item -> block.  Sequence b owns the items from cu[b] / 16 + 2 b on: n
// tokens touch at most n / 16 + 2 blocks, so the owners' ranges never overlap
// and an item finds its sequence by counting the starts at or below it (all
// threads at once).  Items past a sequence's blocks have nothing to do.
template <int NT>
__device__ __forceinline__ bool find_span(const BlockRaggedParams& r, int item, int tid, Span& s) {
  int b = item, t0 = item, t1 = item + 1, base = item;
  if (r.cu != nullptr) {
    int count = 0;
    for (int b0 = 0; b0 < r.B; b0 += NT) {
      const int i = b0 + tid;
      if (item == 0 && i < r.B && (r.cu[i] < 0 || r.cu[i] > r.cu[i + 1] || r.cu[i + 1] > r.T)) record_error(2);
      count += __syncthreads_count(i < r.B && (long long)(r.cu[i] >> 4) + 2ll * i <= item);
    }
    b = count - 1;
    if (b < 0) return false;
    t0 = r.cu[b];
    t1 = r.cu[b + 1];
    base = (t0 >> 4) + 2 * b;
  }
  const int L = r.seq_lens[b];
  if (r.cu == nullptr && L <= 0) return false;  // an empty slot of a padded batch
  if (t0 == t1) return false;
  const bool ok = t0 >= 0 && t1 > t0 && t1 <= r.T && L >= t1 - t0 && (L - 1) / kBS < r.max_blocks;
  if (!ok) {
    if (tid == 0) record_error(2);
    return false;
  }
  const int first = L - (t1 - t0);
  const int lb = (first >> 4) + (item - base);
  if (lb > ((L - 1) >> 4)) return false;
  s.phys = r.block_tables[(size_t)b * r.max_blocks + lb];
  if (s.phys < 0 || s.phys >= r.num_blocks) {
    if (tid == 0) record_error(2);
    return false;
  }
  s.f = max(0, first - lb * kBS);
  s.e = min(kBS, L - lb * kBS);
  s.tok0 = t0 + lb * kBS - first;
  return true;
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ int byte_of(uint32_t w, int i) { return (int)(int8_t)((w >> (8 * i)) & 0xffu); }
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes (low bytes of q) of N values under the block's scale.
template <int N>
__device__ __forceinline__ void quantize(const float (&x)[N], float s, float y, uint32_t (&q)[N]) {
  if (s > 0.f) {
    div_rne_row(x, s, y, q);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = 0u;
  }
}

// Four codes of an older token brought to the grown scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = rne_bits(__fmul_rn((float)byte_of(w, i), ratio));
  return pack4(q[0], q[1], q[2], q[3]);
}

template <int D>
__global__ void __launch_bounds__(D) block_kv_write_kernel(BlockRaggedParams r, BlockWriteParams p) {
  constexpr int H = D / 2;         // threads per page
  constexpr int WS = D / 64;       // warps per page
  __shared__ float s_amax[2 * WS];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, h = blockIdx.y;
  Span s;
  if (!find_span<D>(r, blockIdx.x, tid, s)) return;  // the same answer in every thread
  const bool vside = tid >= H;
  const int st = vside ? tid - H : tid;
  const size_t page = ((size_t)s.phys * r.Hkv + h) * (D * kBS);
  float* scale = (vside ? p.v_scale : p.k_scale) + (size_t)s.phys * r.Hkv + h;
  const float s_old = s.f > 0 ? *scale : 0.f;
  const bool keep = s.f > 0 || s.e < kBS;  // a part of the page stays
  float amax = 0.f;
  // K: 16-dim chunks of one token, two per thread, neighbours along the row.
  uint4 kx[2][2], ko[2];
  int kc[2], kt[2];
  // V: four dims of eight tokens (half a row of the page each).
  const int dq = st % (D / 4), half = st / (D / 4);
  uint2 vx[8], vo[4];
  if (!vside) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int id = j * H + st;
      kc[j] = id % (D / 16);
      kt[j] = id / (D / 16);
      kx[j][0] = kx[j][1] = ko[j] = make_uint4(0, 0, 0, 0);
      if (kt[j] >= s.f && kt[j] < s.e) {
        const uint4* src = reinterpret_cast<const uint4*>(p.k + (int64_t)(s.tok0 + kt[j]) * p.k_stride + h * D + kc[j] * 16);
        kx[j][0] = __ldg(src);
        kx[j][1] = __ldg(src + 1);
      } else if (kt[j] < s.f) {
        ko[j] = *reinterpret_cast<const uint4*>(p.k_cache + page + (kc[j] * kBS + kt[j]) * 16);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {kx[j][i].x, kx[j][i].y, kx[j][i].z, kx[j][i].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) amax = fmaxf(amax, fmaxf(fabsf(lo_bf16(w[u])), fabsf(hi_bf16(w[u]))));
      }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = half * 8 + i;
      vx[i] = make_uint2(0, 0);
      if (t >= s.f && t < s.e)
        vx[i] = __ldg(reinterpret_cast<const uint2*>(p.v + (int64_t)(s.tok0 + t) * p.v_stride + h * D + dq * 4));
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      vo[d] = keep ? *reinterpret_cast<const uint2*>(p.v_cache + page + (dq * 4 + d) * kBS + half * 8) : make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      amax = fmaxf(amax, fmaxf(fmaxf(fabsf(lo_bf16(vx[i].x)), fabsf(hi_bf16(vx[i].x))),
                               fmaxf(fabsf(lo_bf16(vx[i].y)), fabsf(hi_bf16(vx[i].y)))));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
  __syncthreads();  // also: every read of the old scale is done
  amax = 0.f;
#pragma unroll
  for (int w = 0; w < WS; ++w) amax = fmaxf(amax, s_amax[(vside ? WS : 0) + w]);
  const float sn = fmaxf(s_old, div127(amax));
  const float y = __frcp_rn(sn);
  const bool grow = s.f > 0 && sn != s_old;
  const float ratio = grow ? __fdiv_rn(s_old, sn) : 1.f;
  if (st == 0 && (s.f == 0 || grow)) *scale = sn;
  if (!vside) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint4* dst = reinterpret_cast<uint4*>(p.k_cache + page + (kc[j] * kBS + kt[j]) * 16);
      if (kt[j] >= s.f && kt[j] < s.e) {
        const uint32_t w[8] = {kx[j][0].x, kx[j][0].y, kx[j][0].z, kx[j][0].w,
                               kx[j][1].x, kx[j][1].y, kx[j][1].z, kx[j][1].w};
        float x[16];
        uint32_t q[16];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          x[2 * u] = lo_bf16(w[u]);
          x[2 * u + 1] = hi_bf16(w[u]);
        }
        quantize(x, sn, y, q);
        *dst = make_uint4(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]), pack4(q[8], q[9], q[10], q[11]),
                          pack4(q[12], q[13], q[14], q[15]));
      } else if (grow && kt[j] < s.f) {
        *dst = make_uint4(rescale4(ko[j].x, ratio), rescale4(ko[j].y, ratio), rescale4(ko[j].z, ratio),
                          rescale4(ko[j].w, ratio));
      }
    }
  } else if (s.f < half * 8 + 8 && (s.e > half * 8 || grow)) {
    // some byte of this half row changes: new tokens, or older ones under a grown scale
    float x[32];
    uint32_t q[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[4 * i] = lo_bf16(vx[i].x);
      x[4 * i + 1] = hi_bf16(vx[i].x);
      x[4 * i + 2] = lo_bf16(vx[i].y);
      x[4 * i + 3] = hi_bf16(vx[i].y);
    }
    quantize(x, sn, y, q);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t out[2];
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t old = w ? vo[d].y : vo[d].x;
        const uint32_t neu = pack4(q[16 * w + d], q[16 * w + 4 + d], q[16 * w + 8 + d], q[16 * w + 12 + d]);
        const uint32_t res = grow ? rescale4(old, ratio) : old;
        uint32_t m_new = 0, m_res = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = half * 8 + 4 * w + i;
          if (t < s.f) m_res |= 0xffu << (8 * i);
          else if (t < s.e) m_new |= 0xffu << (8 * i);
        }
        out[w] = (neu & m_new) | (res & m_res) | (old & ~(m_new | m_res));
      }
      *reinterpret_cast<uint2*>(p.v_cache + page + (dq * 4 + d) * kBS + half * 8) = make_uint2(out[0], out[1]);
    }
  } else if (grow && half * 8 < s.f) {
    // a half row of older tokens only
#pragma unroll
    for (int d = 0; d < 4; ++d)
      *reinterpret_cast<uint2*>(p.v_cache + page + (dq * 4 + d) * kBS + half * 8) =
          make_uint2(rescale4(vo[d].x, ratio), rescale4(vo[d].y, ratio));
  }
}

// ---- reading back: value = RN(code * scale), fp32 or rounded to bf16 (RNE).
template <bool BF>
__device__ __forceinline__ void store4(void* out, size_t i, float a, float b, float c, float d) {
  if constexpr (BF)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) = make_uint2(bf16x2_rn(a, b), bf16x2_rn(c, d));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = make_float4(a, b, c, d);
}

template <int D, bool BF>
__global__ void __launch_bounds__(D) block_kv_read_kernel(BlockRaggedParams r, BlockReadParams p) {
  constexpr int H = D / 2;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, h = blockIdx.y;
  Span s;
  if (!find_span<D>(r, blockIdx.x, tid, s)) return;
  const size_t page = ((size_t)s.phys * r.Hkv + h) * (D * kBS);
  if (tid < H) {
    const float sc = p.k_scale[(size_t)s.phys * r.Hkv + h];
    uint4 c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int id = j * H + tid, ch = id % (D / 16), t = id / (D / 16);
      if (t >= s.f && t < s.e) c[j] = *reinterpret_cast<const uint4*>(p.k_cache + page + (ch * kBS + t) * 16);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int id = j * H + tid, ch = id % (D / 16), t = id / (D / 16);
      if (t >= s.f && t < s.e) {
        const size_t o = ((size_t)(s.tok0 + t) * r.Hkv + h) * D + ch * 16;
        const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __fmul_rn((float)byte_of(w[i >> 2], i & 3), sc);
        if constexpr (BF) {  // 16-byte stores
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k_out) + o);
          dst[0] = make_uint4(bf16x2_rn(x[0], x[1]), bf16x2_rn(x[2], x[3]), bf16x2_rn(x[4], x[5]), bf16x2_rn(x[6], x[7]));
          dst[1] = make_uint4(bf16x2_rn(x[8], x[9]), bf16x2_rn(x[10], x[11]), bf16x2_rn(x[12], x[13]),
                              bf16x2_rn(x[14], x[15]));
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 4) store4<false>(p.k_out, o + i, x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
      }
    }
  } else {
    const int st = tid - H, dq = st % (D / 4), half = st / (D / 4);
    if (s.f >= half * 8 + 8 || s.e <= half * 8) return;
    const float sc = p.v_scale[(size_t)s.phys * r.Hkv + h];
    uint2 c[4];
#pragma unroll
    for (int d = 0; d < 4; ++d)
      c[d] = *reinterpret_cast<const uint2*>(p.v_cache + page + (dq * 4 + d) * kBS + half * 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = half * 8 + i;
      if (t >= s.f && t < s.e) {
        float x[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) x[d] = __fmul_rn((float)byte_of(i < 4 ? c[d].x : c[d].y, i & 3), sc);
        store4<BF>(p.v_out, ((size_t)(s.tok0 + t) * r.Hkv + h) * D + dq * 4, x[0], x[1], x[2], x[3]);
      }
    }
  }
}

dim3 ragged_grid(const BlockRaggedParams& r) {
  return dim3(r.cu == nullptr ? r.B : r.T / kBS + 2 * r.B, r.Hkv);
}

}  // namespace

cudaError_t launch_block_kv_write(const BlockRaggedParams& r, const BlockWriteParams& p, cudaStream_t stream) {
  const dim3 grid = ragged_grid(r);
  if (r.D == 256) return launch_pdl(block_kv_write_kernel<256>, grid, dim3(256), 0, stream, r, p);
  if (r.D == 128) return launch_pdl(block_kv_write_kernel<128>, grid, dim3(128), 0, stream, r, p);
  return launch_pdl(block_kv_write_kernel<64>, grid, dim3(64), 0, stream, r, p);
}

cudaError_t launch_block_kv_read(const BlockRaggedParams& r, const BlockReadParams& p, cudaStream_t stream) {
  const dim3 grid = ragged_grid(r);
  if (p.out_bf16) {
    if (r.D == 256) return launch_pdl(block_kv_read_kernel<256, true>, grid, dim3(256), 0, stream, r, p);
    if (r.D == 128) return launch_pdl(block_kv_read_kernel<128, true>, grid, dim3(128), 0, stream, r, p);
    return launch_pdl(block_kv_read_kernel<64, true>, grid, dim3(64), 0, stream, r, p);
  }
  if (r.D == 256) return launch_pdl(block_kv_read_kernel<256, false>, grid, dim3(256), 0, stream, r, p);
  if (r.D == 128) return launch_pdl(block_kv_read_kernel<128, false>, grid, dim3(128), 0, stream, r, p);
  return launch_pdl(block_kv_read_kernel<64, false>, grid, dim3(64), 0, stream, r, p);
}

}  // namespace i8kv
