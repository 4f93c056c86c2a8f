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
// One block of threads owns a cache block and head (K and V) -- a cluster of
// up to eight where the cache block has more slots than its registers hold --
// so nothing is shared between blocks of threads and the bits do not depend on
// their order.  A thread has P pieces (16 elements of a token's row, rope.cuh)
// in registers from the load to the store and works out the eight sines and
// cosines of its own pairs once for the heads that it goes through: one when
// there are few blocks of threads, all of them when there are many.
// What bounds it: bytes (2 read, 1 written per value) and the latency of one
// pass: table, scales, rows, maxima, stores, each waiting for the one before.
// 24 prompts of up to 1024 tokens, 16 query and 4 KV heads of 128, 64-token
// blocks: 36 to 38 us, 2.9 TB/s; a token for each of 64 sequences: 6 us.
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
  // Blocks of threads for K/V; those for the queries follow.  (Dealt evenly
  // over the grid instead: 44 us for the call that takes 36.)
  int64_t kv_blocks;
  int cluster;           // of them per cache block and head group
  int heads;             // heads that one goes through
  int64_t groups;        // upper bound of the touched cache blocks
};

// The cache block that group x stands for.  n new tokens touch at most
// floor((n + bs - 2) / bs) + 1 cache blocks: dense, that many groups a
// sequence; packed, sequence b owns the groups from floor(start_b / bs) + 2 b
// on, floor(n_b / bs) + 2 at least.
struct TouchedBlock {
  int b, start, n;   // sequence, its first new token in the call, their count
  int64_t first;     // position of the block's slot 0
  int64_t pos0;      // position of the sequence's first new token
  int64_t blk;       // cache block, -1: nothing to do
};

__host__ __device__ inline int64_t dense_groups(int n, int block_shift) {
  return ((static_cast<int64_t>(n) + (int64_t{1} << block_shift) - 2) >> block_shift) + 1;
}

__device__ __forceinline__ int64_t group_base(const RopeParams &r, int b) {
  if (!r.cu) return static_cast<int64_t>(b) * dense_groups(r.n, r.block_shift);
  return (max(__ldg(r.cu + b), 0) >> r.block_shift) + 2 * static_cast<int64_t>(b);
}

__device__ __forceinline__ TouchedBlock touched_block(const RopeParams &r, int64_t x) {
  TouchedBlock k{};
  k.blk = -1;
  int lo = 0, hi = r.batch - 1;
  if (!r.cu) lo = hi = static_cast<int>(x / dense_groups(r.n, r.block_shift));
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

// Another block's shared variable, within the cluster.
__device__ __forceinline__ int cluster_ld(const int *v, uint32_t rank) {
  uint32_t a;
  int r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(v)), "r"(rank));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Slots [part * S, (part + 1) * S) of the cache block of group x, KV heads head0
// .. head0 + p.heads - 1; S = P * kRopeThreads / (2 U) rows of K and as many of V.
constexpr int kAppendHeads = 8;  // heads per block of threads at most

template <int P>
__device__ __forceinline__ void append_block_q8(const AppendQ8Params &p, int64_t x, int head0, int part) {
  __shared__ TouchedBlock s_blk;
  __shared__ int s_max[kAppendHeads][2];
  const RopeParams &r = p.r;
  const int tid = threadIdx.x, U = r.D >> 4, u = tid & (U - 1);
  if (tid == 0) s_blk = touched_block(r, x);
  if (tid < 2 * kAppendHeads) s_max[tid >> 1][tid & 1] = 0;
  __syncthreads();
  const TouchedBlock B = s_blk;
  if (B.blk < 0) return;  // uniform over the cluster
  const int bs = 1 << r.block_shift;
  const int slot0 = static_cast<int>(max(B.pos0 - B.first, int64_t{0}));
  const int slot1 = static_cast<int>(min(B.pos0 + B.n - B.first, static_cast<int64_t>(bs)));
  const int t0 = static_cast<int>(B.first - B.pos0);  // token of slot 0
  const int per_pass = kRopeThreads / U, S = P * per_pass / 2;
  const bool turns = p.rotate && 16 * u < 2 * r.f.half;
  const int2 kch = p.rotate ? piece_chunks(r.f, u) : make_int2(2 * u, 2 * u + 1);
  // piece k: row i of the S K rows, then the S V rows
  auto row_of = [&](int k, int &w, int &slot) {
    const int i = tid / U + k * per_pass;
    w = i >= S ? 1 : 0;
    slot = part * S + i - w * S;
  };
  // the K pieces' cosines and sines (the first half of the pieces; P = 1: the
  // first half of the threads)
  constexpr int kTurn = P > 1 ? P / 2 : 1;
  float2 cs[kTurn][8];
#pragma unroll
  for (int k = 0; k < kTurn; ++k) {
    int w, slot;
    row_of(k, w, slot);
    if (w == 0 && turns && slot >= slot0 && slot < slot1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[k][e] = rope_cs(r.f, static_cast<int>(B.first + slot), 8 * u + e);
    }
  }
  const int heads = min(p.heads, p.Hkv - head0);
  for (int hh = 0; hh < heads; ++hh) {
    const int head = head0 + hh;
    uint4 a[P], b[P];
#pragma unroll
    for (int k = 0; k < P; ++k) {
      int w, slot;
      row_of(k, w, slot);
      a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
      if (slot >= slot0 && slot < slot1) {
        const RopeRows &X = p.kv[w];
        const uint4 *s = reinterpret_cast<const uint4 *>(
            X.src + (r.cu ? 0 : B.b * X.s0) + (static_cast<int64_t>(B.start) + t0 + slot) * X.s1 + head * X.s2);
        const int2 c = w ? make_int2(2 * u, 2 * u + 1) : kch;
        a[k] = __ldg(s + c.x);  // (never written here)
        b[k] = __ldg(s + c.y);
      }
    }
    // (the old scales are fetched beside them)
    int old[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (slot0 > 0) old[w] = p.scale[w][B.blk * p.s0[w] + head * p.s1[w]];
    float v[P][16];
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < P; ++k) {
      int w, slot;
      row_of(k, w, slot);
      if (k < kTurn && w == 0 && turns && slot >= slot0 && slot < slot1) {
        turn_piece(r.f, cs[k < kTurn ? k : 0], a[k], b[k], v[k]);
      } else {
        const uint32_t wa[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[k][2 * e] = bf_lo(wa[e]);
          v[k][2 * e + 1] = bf_hi(wa[e]);
        }
      }
      float m = 0.f;  // (finite values: an infinity saturates)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float y = fabsf(v[k][e]);
        m = fmaxf(m, y < __int_as_float(0x7f800000) ? y : 0.f);
      }
      if (w) top[1] = fmaxf(top[1], m); else top[0] = fmaxf(top[0], m);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // non-negative floats are ordered like their bits
      const int m = __reduce_max_sync(0xffffffffu, __float_as_int(top[w]));
      if ((tid & 31) == 0 && m) atomicMax(&s_max[hh][w], m);
    }
    // the maxima are complete, and every thread has read the old scales
    int all[2] = {0, 0};
    if (p.cluster > 1) {
      cluster_sync();
      for (int c = 0; c < p.cluster; ++c)
#pragma unroll
        for (int w = 0; w < 2; ++w) all[w] = max(all[w], cluster_ld(&s_max[hh][w], c));
    } else {
      __syncthreads();
      all[0] = s_max[hh][0];
      all[1] = s_max[hh][1];
    }
    int byte[2];
    float lift[2] = {1.f, 1.f};  // factor of the earlier tokens, 1: as they are
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      byte[w] = need_byte(__int_as_float(all[w]));
      if (slot0 > 0) {
        if (old[w] < kScaleByteMin || old[w] > kScaleByteMax) {
          if (tid == 0 && part == 0 && r.err) atomicOr(r.err, kErrScale);
          old[w] = min(max(old[w], kScaleByteMin), kScaleByteMax);
        }
        byte[w] = max(old[w], byte[w]);
        lift[w] = __int_as_float((127 - min(byte[w] - old[w], 126)) << 23);
      }
    }
    if (part == 0 && tid < 2)
      p.scale[tid][B.blk * p.s0[tid] + head * p.s1[tid]] = static_cast<uint8_t>(tid ? byte[1] : byte[0]);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      int w, slot;
      row_of(k, w, slot);
      uint8_t *row = p.cache[w] + B.blk * p.c0[w] + slot * p.c1[w] + head * p.c2[w];
      if (slot >= slot0 && slot < slot1) {
        store_piece(row, w ? make_int2(2 * u, 2 * u + 1) : kch, v[k], inv_scale_of(w ? byte[1] : byte[0]));
      } else if (slot < slot0 && (w ? lift[1] : lift[0]) != 1.f) {
        // requantise an earlier token
        const float f = w ? lift[1] : lift[0];
        uint4 *q = reinterpret_cast<uint4 *>(row) + u;
        const uint4 z = *q;
        uint32_t o[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c = __half22float2(half2_of_e4m3x2(o[e] & 0xFFFFu));
          const float2 d = __half22float2(half2_of_e4m3x2(o[e] >> 16));
          o[e] = e4m3x2_of(__fmul_rn(c.x, f), __fmul_rn(c.y, f)) |
                 (e4m3x2_of(__fmul_rn(d.x, f), __fmul_rn(d.y, f)) << 16);
        }
        *q = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (p.cluster > 1) cluster_sync();  // the others have read this block's maxima
}

template <int P>
__global__ void __launch_bounds__(kRopeThreads, 4)
    append_q8_kernel(const __grid_constant__ AppendQ8Params p) {
  __shared__ __align__(16) float2 cs[kRopeWarps][64];
  const int64_t x = blockIdx.x;
  if (x < p.kv_blocks) {
    const int64_t y = x / p.cluster;
    const int per = (p.Hkv + p.heads - 1) / p.heads;  // head groups
    append_block_q8<P>(p, y / per, static_cast<int>(y % per) * p.heads, static_cast<int>(x % p.cluster));
  } else if (p.r.cu && x == gridDim.x - 1) {
    check_ranges(p.r);  // (a block of its own, behind the queries')
  } else if (p.r.x[0].heads > 0) {
    const int warp = threadIdx.x >> 5;
    rope_warp(p.r, (x - p.kv_blocks) * kRopeWarps + warp, cs[warp]);
  }
}

}  // namespace pkv
