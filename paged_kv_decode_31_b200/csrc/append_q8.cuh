// append_q8.cuh -- new K/V tokens into an 8-bit paged cache, the keys (and the
// queries beside them) rotated on the way.
//
// A block of the cache and a KV head share one scale 2^e, for K and for V.
// For every block that the new tokens touch:
//   a    = max |x| over its new tokens (K after the rotation, in fp32),
//   need = the least e with a <= 448 2^e, held to [kScaleExpMin, kScaleExpMax],
//   e'   = max(e, need) when the block holds earlier tokens, else need;
//   the earlier tokens become e4m3(q 2^(e - e')) when e' > e, and the new ones
//   e4m3(x 2^-e').
// Scales are powers of two so that raising one only shifts exponents: an
// earlier value keeps its bits unless it becomes subnormal, and a block filled
// token by token is not rounded again at every step.
//
// One block of threads owns a cache block and head (K and V), so nothing is
// shared between blocks of threads and the bits do not depend on their order.
// A thread takes a 16-element piece of a token's row (rope.cuh) and works out
// the eight sines and cosines of its own pairs: each is used once per head.
// What bounds it: bytes (2 read, 1 written per value).
#pragma once

#include "f8.cuh"
#include "rope.cuh"

namespace pkv {

struct AppendQ8Params {
  RopeParams r;          // queries, frequencies, token layout and block table
  RopeRows kv[2];        // k_new, v_new (src)
  uint8_t *cache[2];     // K, V: e4m3, strides (block, slot, head)
  int64_t c0[2], c1[2], c2[2];
  uint8_t *scale[2];     // scale bytes, strides (block, head)
  int64_t s0[2], s1[2];
  int Hkv;
  int rotate;
  int64_t kv_blocks;     // blocks of threads for K/V; those for the queries follow
  int64_t groups;        // upper bound of the touched cache blocks
};

// The cache block that group x stands for: sequence b owns the groups from
// floor(start_b / bs) + 2 b on, at least as many as its new tokens can touch
// (floor(n_b / bs) + 2).
struct TouchedBlock {
  int b, start, n;   // sequence, its first new token in the call, their count
  int64_t first;     // position of the block's slot 0
  int64_t pos0;      // position of the sequence's first new token
  int64_t blk;       // cache block, -1: nothing to do
};

__device__ __forceinline__ int64_t group_base(const RopeParams &r, int b) {
  const int64_t start = r.cu ? max(__ldg(r.cu + b), 0) : static_cast<int64_t>(b) * r.n;
  return (start >> r.block_shift) + 2 * static_cast<int64_t>(b);
}

__device__ __forceinline__ TouchedBlock touched_block(const RopeParams &r, int64_t x) {
  TouchedBlock k{};
  k.blk = -1;
  int lo = 0, hi = r.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (group_base(r, mid) <= x) lo = mid; else hi = mid - 1;
  }
  k.b = lo;
  const int64_t j = x - group_base(r, lo);
  if (r.cu) {
    const int2 a = packed_range(r.cu, lo, r.tokens, r.err);
    k.start = a.x;
    k.n = a.y;
  } else {
    k.start = 0;
    k.n = r.n;
  }
  if (k.n <= 0 || j < 0) return k;
  k.pos0 = __ldg(r.seqlens + lo);
  const int64_t col = (k.pos0 >> r.block_shift) + j;
  if (k.pos0 < 0) {
    if (r.err) atomicOr(r.err, kErrTableWidth);
    return k;
  }
  if (col > (k.pos0 + k.n - 1) >> r.block_shift) return k;
  if (col >= r.max_blocks_per_seq) {
    if (r.err) atomicOr(r.err, kErrTableWidth);
    return k;
  }
  k.first = col << r.block_shift;
  const int32_t blk = __ldg(r.block_table + lo * r.bt_stride + col);
  if (blk < 0 || blk >= r.num_blocks) {
    if (r.err) atomicOr(r.err, kErrBadBlock);
    return k;
  }
  k.blk = blk;
  return k;
}

// The least exponent e with a <= 448 * 2^e, as a scale byte (a finite, >= 0).
__device__ __forceinline__ int need_byte(float a) {
  // a = f 2^x with f in [1, 2): 448 = 1.75 * 2^8, so e = x - 8, one more when f > 1.75
  const uint32_t w = __float_as_uint(a);
  const int byte = static_cast<int>(w >> 23) - 8 + ((w & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(byte, kScaleByteMin), kScaleByteMax);  // (subnormal a: far below the range)
}

// 16 values (a piece's two chunks) to e4m3 under 2^(127 - byte).
__device__ __forceinline__ void store_piece(uint8_t *row, int2 ch, const float (&v)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    w[e] = e4m3x2_of(__fmul_rn(v[4 * e], inv), __fmul_rn(v[4 * e + 1], inv)) |
           (e4m3x2_of(__fmul_rn(v[4 * e + 2], inv), __fmul_rn(v[4 * e + 3], inv)) << 16);
  *reinterpret_cast<uint2 *>(row + ch.x * 8) = make_uint2(w[0], w[1]);
  *reinterpret_cast<uint2 *>(row + ch.y * 8) = make_uint2(w[2], w[3]);
}

__device__ __forceinline__ void append_block_q8(const AppendQ8Params &p, int64_t x, int head) {
  __shared__ TouchedBlock s_blk;
  __shared__ int s_max[2];
  const RopeParams &r = p.r;
  const int tid = threadIdx.x, U = r.D >> 4, u = tid % U;
  if (tid == 0) s_blk = touched_block(r, x);
  if (tid < 2) s_max[tid] = 0;
  __syncthreads();
  const TouchedBlock B = s_blk;
  if (B.blk < 0) return;  // uniform
  const int bs = 1 << r.block_shift;
  const int slot0 = static_cast<int>(max(B.pos0 - B.first, int64_t{0}));
  const int slot1 = static_cast<int>(min(B.pos0 + B.n - B.first, static_cast<int64_t>(bs)));
  const int n_new = slot1 - slot0;
  const int t0 = static_cast<int>(B.first + slot0 - B.pos0);  // token of the first one
  // (K rows, then V rows) x U pieces over the block's threads
  const int per_pass = kRopeThreads / U;
  const bool turns = p.rotate && 16 * u < 2 * r.f.half;
  const int2 ch = p.rotate ? piece_chunks(r.f, u) : make_int2(2 * u, 2 * u + 1);
  auto load = [&](int i, float (&v)[16]) {
    const int w = i >= n_new ? 1 : 0, t = t0 + i - w * n_new;
    const RopeRows &X = p.kv[w];
    const uint16_t *s = X.src + (r.cu ? 0 : B.b * X.s0) + (static_cast<int64_t>(B.start) + t) * X.s1 +
                        head * X.s2;
    const int2 c = w ? make_int2(2 * u, 2 * u + 1) : ch;
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(s) + c.x);  // (never written here)
    const uint4 b = __ldg(reinterpret_cast<const uint4 *>(s) + c.y);
    if (w == 0 && turns) {
      float2 cs[8];
      const int pos = static_cast<int>(B.pos0 + t);
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = rope_cs(r.f, pos, 8 * u + e);
      turn_piece(r.f, cs, a, b, v);
    } else {
      const uint32_t wa[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[2 * e] = bf_lo(wa[e]);
        v[2 * e + 1] = bf_hi(wa[e]);
      }
    }
  };
  // pass 1: the largest magnitudes (finite ones: an infinity saturates)
  float v[16];
  float top[2] = {0.f, 0.f};
  for (int i = tid / U; i < 2 * n_new; i += per_pass) {
    load(i, v);
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = fabsf(v[e]);
      m = fmaxf(m, y < __int_as_float(0x7f800000) ? y : 0.f);
    }
    if (i >= n_new) top[1] = fmaxf(top[1], m); else top[0] = fmaxf(top[0], m);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    // non-negative floats are ordered like their bits
    const int m = __reduce_max_sync(0xffffffffu, __float_as_int(top[w]));
    if ((tid & 31) == 0) atomicMax(&s_max[w], m);
  }
  __syncthreads();
  int byte[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint8_t *sp = p.scale[w] + B.blk * p.s0[w] + head * p.s1[w];
    const int need = need_byte(__int_as_float(s_max[w]));
    byte[w] = need;
    if (slot0 > 0) {
      int old = *sp;
      if (old < kScaleByteMin || old > kScaleByteMax) {
        if (tid == 0 && r.err) atomicOr(r.err, kErrScale);
        old = min(max(old, kScaleByteMin), kScaleByteMax);
      }
      byte[w] = max(old, need);
      if (byte[w] > old) {
        // requantise the earlier tokens
        const float f = __int_as_float((127 - min(byte[w] - old, 126)) << 23);
        for (int i = tid / U; i < slot0; i += per_pass) {
          uint4 *q = reinterpret_cast<uint4 *>(p.cache[w] + B.blk * p.c0[w] + i * p.c1[w] +
                                               head * p.c2[w]) + u;
          const uint4 z = *q;
          uint32_t o[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = __half22float2(half2_of_e4m3x2(o[e] & 0xFFFFu));
            const float2 b = __half22float2(half2_of_e4m3x2(o[e] >> 16));
            o[e] = e4m3x2_of(__fmul_rn(a.x, f), __fmul_rn(a.y, f)) |
                   (e4m3x2_of(__fmul_rn(b.x, f), __fmul_rn(b.y, f)) << 16);
          }
          *q = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
  }
  // pass 2: the new tokens
  for (int i = tid / U; i < 2 * n_new; i += per_pass) {
    load(i, v);
    const int w = i >= n_new ? 1 : 0, slot = slot0 + i - w * n_new;
    uint8_t *row = p.cache[w] + B.blk * p.c0[w] + slot * p.c1[w] + head * p.c2[w];
    store_piece(row, w ? make_int2(2 * u, 2 * u + 1) : ch, v, inv_scale_of(byte[w]));
  }
  __syncthreads();  // every thread has read the old scale
  if (tid < 2) p.scale[tid][B.blk * p.s0[tid] + head * p.s1[tid]] = static_cast<uint8_t>(tid ? byte[1] : byte[0]);
}

__global__ void __launch_bounds__(kRopeThreads)
    append_q8_kernel(const __grid_constant__ AppendQ8Params p) {
  const int64_t x = blockIdx.x;
  if (x < p.kv_blocks) {
    append_block_q8(p, x / p.Hkv, static_cast<int>(x % p.Hkv));
  } else {
    const int64_t first = (x - p.kv_blocks) * p.r.per_block;
    const int64_t left = p.r.tokens - first;
    rope_tokens(p.r, first, static_cast<int>(left < p.r.per_block ? left : p.r.per_block));
  }
}

}  // namespace pkv
