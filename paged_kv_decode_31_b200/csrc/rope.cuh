// rope.cuh -- rotary positions, alone and on the way into a paged cache.
//
// Pair i (0 <= i < r / 2, r = the rotated part of the head) of a row at
// position p turns by theta = p f_i:
//   y1 = x1 c - x2 s,  y2 = x2 c + x1 s,  c = m cos theta, s = m sin theta
// with (x1, x2) the elements (i, i + r / 2) (half layout) or (2i, 2i + 1)
// (interleaved); elements past r are copied.  The transpose (s negated) is the
// gradient.  theta is formed in fp64 and reduced to a fraction of a turn there
// (p f_i reaches 10^6 radians, where fp32 angles are off by 0.06), the
// fraction's sine and cosine are fp32 (sincospif), y is rounded to bf16 once.
//
// What bounds it: bytes.  A row is read and written once and the arithmetic is
// 3 operations per element.  A warp takes kRopePasses passes of rows of one
// token (12 rows at head_dim 128), all their loads in flight before the
// position's table look-up and the sines, which it works out once for them; no
// barrier, so that one warp's look-ups hide behind the rows of others (blocks
// of four tokens that shared the sines through barriers: 52 us for 16389
// tokens of 20 heads, 168 MB).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "contract.cuh"
#include "packed.cuh"
#include "ptx.cuh"

namespace pkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// Rows a lane has in flight at most: 3 leave four blocks of threads per SM
// (16389 tokens of 20 heads: 1: 37 us, 2: 32, 3: 29, 4: 36).
constexpr int kRopePasses = 3;

struct RopeFreq {
  const float *inv_freq;  // [half]
  int half;               // r / 2, a multiple of 8
  int interleaved;
  float mscale;
  float sign;             // +1, or -1 for the transpose
};

// Heads of one tensor, from src to dst.  Dense side: element strides (batch,
// token, head); paged side: (block, slot, head).
struct RopeRows {
  const uint16_t *src;
  uint16_t *dst;
  int64_t s0, s1, s2, d0, d1, d2;
  int heads;
  int rotate;
};

struct RopeParams {
  RopeFreq f;
  RopeRows x[3];  // queries, keys, values (heads = 0: absent)
  int src_paged, dst_paged;  // of x[1] and x[2]
  int D;
  // the tokens: dense [batch, n], or packed (cu != null, n unused)
  int64_t tokens;
  int batch, n;
  const int32_t *cu;
  // positions: one per token, or seqlens[b] + t with the cache's block table
  const int32_t *positions;
  const int32_t *seqlens;
  const int32_t *block_table;
  int64_t bt_stride, num_blocks;
  int max_blocks_per_seq, block_shift;
  int chunks, passes;  // warps per token, passes of rows in each
  int32_t *err;
};

__device__ __forceinline__ float2 rope_cs(const RopeFreq &f, int pos, int i) {
  double t = static_cast<double>(pos) * static_cast<double>(__ldg(f.inv_freq + i)) *
             0.15915494309189533577;  // turns: 1 / (2 pi)
  t -= rint(t);
  float s, c;
  sincospif(2.f * static_cast<float>(t), &s, &c);
  return make_float2(__fmul_rn(c, f.mscale), __fmul_rn(s, __fmul_rn(f.mscale, f.sign)));
}

__device__ __forceinline__ float2 turned(float x1, float x2, float2 cs) {
  return make_float2(__fmaf_rn(x1, cs.x, -__fmul_rn(x2, cs.y)),
                     __fmaf_rn(x2, cs.x, __fmul_rn(x1, cs.y)));
}

// A row is D / 16 pieces of 32 bytes, two 16-byte chunks each, and a piece
// holds both sides of its pairs: piece u < r / 16 turns pairs 8u .. 8u + 7.
// Chunk indexes of piece u:
__device__ __forceinline__ int2 piece_chunks(const RopeFreq &f, int u) {
  if (!f.interleaved) {
    const int h = f.half >> 3;
    if (u < h) return make_int2(u, u + h);
  }
  return make_int2(2 * u, 2 * u + 1);  // (past r the chunks 2u, 2u + 1 are the copied ones)
}

__device__ __forceinline__ uint32_t bf2_of(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// The eight pairs of a rotated piece (a, b: its chunks) in fp32, element
// order kept: v[0..7] = chunk a, v[8..15] = chunk b.
__device__ __forceinline__ void turn_piece(const RopeFreq &f, const float2 (&cs)[8], uint4 a, uint4 b,
                                           float (&v)[16]) {
  const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
  if (f.interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = turned(bf_lo(wa[e]), bf_hi(wa[e]), cs[e]);
      const float2 z = turned(bf_lo(wb[e]), bf_hi(wb[e]), cs[4 + e]);
      v[2 * e] = y.x;
      v[2 * e + 1] = y.y;
      v[8 + 2 * e] = z.x;
      v[8 + 2 * e + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y = turned(bf_lo(wa[e]), bf_lo(wb[e]), cs[2 * e]);
      const float2 z = turned(bf_hi(wa[e]), bf_hi(wb[e]), cs[2 * e + 1]);
      v[2 * e] = y.x;
      v[2 * e + 1] = z.x;
      v[8 + 2 * e] = y.y;
      v[8 + 2 * e + 1] = z.y;
    }
  }
}

// What a warp needs to know of its token.
struct RopeToken {
  int pos;
  int ok;       // the token exists
  int in_cache; // its cache row exists (paged calls)
  int64_t b, t; // dense coordinates (packed: b = 0, t = the packed index)
  int64_t blk, slot;
};

// Sequence b's new tokens in the packed axis, held to [0, total): start and
// count.  A range outside it (or decreasing) is reported.
__device__ __forceinline__ int2 packed_range(const int32_t *cu, int b, int64_t total, int32_t *err) {
  const int a = __ldg(cu + b), e = __ldg(cu + b + 1);
  const bool bad = a < 0 || e < a || e > total;
  if (bad && err) atomicOr(err, kErrQueryLen);
  return bad ? make_int2(0, 0) : make_int2(a, e - a);
}

// Every range of a packed call, by the threads of one block.  (The search for a
// token's sequence does not pass by all of them when they do not ascend.)
__device__ __forceinline__ void check_ranges(const RopeParams &p) {
  for (int b = threadIdx.x; b < p.batch; b += kRopeThreads) packed_range(p.cu, b, p.tokens, p.err);
}

__device__ __forceinline__ RopeToken rope_token(const RopeParams &p, int64_t r) {
  RopeToken k{};
  int b, t;
  if (p.cu) {
    b = seq_of_token(p.cu, p.batch, r);
    const int2 a = packed_range(p.cu, b, p.tokens, p.err);
    t = static_cast<int>(r - a.x);
    k.ok = t >= 0 && t < a.y;
    k.b = 0;
    k.t = r;
  } else {
    b = static_cast<int>(r / p.n);
    t = static_cast<int>(r - static_cast<int64_t>(b) * p.n);
    k.ok = 1;
    k.b = b;
    k.t = t;
  }
  if (!k.ok) return k;
  if (p.positions) {
    k.pos = __ldg(p.positions + r);
    return k;
  }
  const int64_t pos = static_cast<int64_t>(__ldg(p.seqlens + b)) + t;
  k.pos = static_cast<int>(pos);
  if (!p.src_paged && !p.dst_paged) return k;
  const int64_t col = pos >> p.block_shift;
  if (pos < 0 || col >= p.max_blocks_per_seq) {
    if (p.err) atomicOr(p.err, kErrTableWidth);
  } else {
    k.blk = __ldg(p.block_table + b * p.bt_stride + col);
    k.slot = pos & ((int64_t{1} << p.block_shift) - 1);
    k.in_cache = k.blk >= 0 && k.blk < p.num_blocks;
    if (!k.in_cache && p.err) atomicOr(p.err, kErrBadBlock);
  }
  return k;
}

// Warp `item` of the call: p.passes passes of 32 / U rows of one token.
// cs: the warp's 64 cosines and sines.
__device__ __forceinline__ void rope_warp(const RopeParams &p, int64_t item, float2 *cs) {
  const int lane = threadIdx.x & 31;
  const int64_t r = item / p.chunks;
  if (r >= p.tokens) return;
  const int U = p.D >> 4, u = lane & (U - 1);  // pieces per row; a lane keeps its piece index
  const int per_pass = 32 / U, h0 = static_cast<int>(item - r * p.chunks) * p.passes * per_pass + lane / U;
  const int2 ch = piece_chunks(p.f, u);
  const bool turns = 16 * u < 2 * p.f.half;
  const int rows = p.x[0].heads + p.x[1].heads + p.x[2].heads;
  const RopeToken T = rope_token(p, r);
  if (!T.ok) return;  // warp-uniform
  uint4 a[kRopePasses], b[kRopePasses];
  uint16_t *dst[kRopePasses];
  bool turn[kRopePasses];
#pragma unroll
  for (int q = 0; q < kRopePasses; ++q) {
    const int h = h0 + q * per_pass;
    dst[q] = nullptr;
    turn[q] = false;
    a[q] = b[q] = make_uint4(0u, 0u, 0u, 0u);
    if (q < p.passes && h < rows) {
      const int w = h < p.x[0].heads ? 0 : h < p.x[0].heads + p.x[1].heads ? 1 : 2;
      const RopeRows &X = p.x[w];
      const int head = h - (w > 0 ? p.x[0].heads : 0) - (w > 1 ? p.x[1].heads : 0);
      const bool sp = w > 0 && p.src_paged, dp = w > 0 && p.dst_paged;
      if (!dp || T.in_cache) {
        dst[q] = X.dst + (dp ? T.blk : T.b) * X.d0 + (dp ? T.slot : T.t) * X.d1 + head * X.d2;
        turn[q] = X.rotate && turns;
        if (!sp || T.in_cache) {  // (otherwise zeros)
          const uint4 *s = reinterpret_cast<const uint4 *>(
              X.src + (sp ? T.blk : T.b) * X.s0 + (sp ? T.slot : T.t) * X.s1 + head * X.s2);
          a[q] = s[ch.x];
          b[q] = s[ch.y];
        }
      }
    }
  }
  for (int i = lane; i < p.f.half; i += 32) cs[i] = rope_cs(p.f, T.pos, i);
  __syncwarp();
  float2 c[8];
  if (turns) {
    const float4 *c4 = reinterpret_cast<const float4 *>(cs + 8 * u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 v = c4[e];
      c[2 * e] = make_float2(v.x, v.y);
      c[2 * e + 1] = make_float2(v.z, v.w);
    }
  }
#pragma unroll
  for (int q = 0; q < kRopePasses; ++q) {
    if (!dst[q]) continue;
    if (turn[q]) {
      float v[16];
      turn_piece(p.f, c, a[q], b[q], v);
      a[q] = make_uint4(bf2_of(v[0], v[1]), bf2_of(v[2], v[3]), bf2_of(v[4], v[5]), bf2_of(v[6], v[7]));
      b[q] = make_uint4(bf2_of(v[8], v[9]), bf2_of(v[10], v[11]), bf2_of(v[12], v[13]), bf2_of(v[14], v[15]));
    }
    reinterpret_cast<uint4 *>(dst[q])[ch.x] = a[q];
    reinterpret_cast<uint4 *>(dst[q])[ch.y] = b[q];
  }
}

// Packed calls have a last block that only looks at the ranges (beside the others:
// no token's rows wait for it).
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float2 cs[kRopeWarps][64];
  if (p.cu && blockIdx.x == gridDim.x - 1) {
    check_ranges(p);
    return;
  }
  const int warp = threadIdx.x >> 5;
  rope_warp(p, static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp, cs[warp]);
}

}  // namespace pkv
