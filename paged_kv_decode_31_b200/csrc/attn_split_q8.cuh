// attn_split_q8.cuh -- split-KV attention over an 8-bit paged cache, few query
// rows per KV head (decode, multi-token decode), sm_100a.
//
// The cache holds K and V as e4m3 values with a scale 2^e for each block of
// tokens and KV head (f8.cuh).  Units, splits, tiles, schedule, roles and the
// merge are those of attn_split.cuh; what differs is the arithmetic of a tile,
// which runs on the 8-bit tensor-core path without ever widening the cache:
//   S^T   = K8 * [q_hi + q_lo]^T   (kind::f8f6f4, M = 128 tokens, N = rows)
//           with the query row taken apart exactly into two 8-bit operands
//           of one scale (split_q), so S is q . k8 to fp32 accumulation;
//   w     = S * (c 2^-k 2^ek) + ev, per token: ek and ev are the exponents of
//           its K and V scales, k the query row's, c = softmax scale * log2 e.
//           w is the base-2 score plus the log of the V scale, so 2^w weighs
//           the token's 8-bit V directly;
//   m     the row's running reference (-inf at the split's start) rises to
//           max(w) - kRefDrop when max(w) > m + 8; P = 2^(w - m) is then at
//           most 2^8 and at least 2^(8 - kRefSlack) for the largest token;
//   O^T  += V8^T * [P_hi | P_mid]^T, P as two 8-bit operands side by side
//           (split_p), joined as O_hi + O_mid / 16 at the split's end;
//   l     = sum of 2^(w - ev - m) = P 2^-ev over the tokens, in fp32.
// (m, l, O) is a partial in the form the merge folds: out = O / l and lse =
// (m + log2 l) ln 2.  Folding the V scale into the exponent keeps every
// operand of one MMA on one scale, whatever the blocks' scales are, and lets
// the reference follow what the tokens contribute to the output.
//
// What bounds it: the cache bytes.  A 128-token tile of one KV head is 32 KB
// (head_dim 128) against 64 KB for bf16, so the softmax chain has half the
// time per tile; with 8-bit operands read in place the tensor cores and the
// shared memory see no conversion traffic (widening the tile to bf16 in shared
// memory would move 5 bytes per cache byte through it).
#pragma once

#include "attn_split.cuh"
#include "f8.cuh"

namespace pkv {

constexpr int kQ8Threads = 512;  // attn_split.cuh's roles, and
constexpr int kPvWarp = 15;      // a second MMA issuer, for P.V

// P <= 2^8 fits e4m3 (448); the reference moves when the largest token passes
// it, and then to 2^kRefDrop below that token, so a row's largest P stays in
// [2^kRefDrop, 2^8] and rescaling O stays rare.
constexpr float kRefTop = 8.f, kRefDrop = 6.f;

struct Q8Params : AttnParams {
  const uint8_t *k_sc, *v_sc;  // scale bytes of (block, KV head)
  int64_t ksc_sb, ksc_sh, vsc_sb, vsc_sh;
  int box_shift;               // log2(box_slots)
};

template <int D, int N, int NS>
struct Q8Cfg {
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static_assert(N == 16 || N == 64, "rows per tile");
  static constexpr int kD = D, kN = N, kNS = NS, kQB = 2;
  static constexpr int kKVBytes = kTileTokens * D;     // one K (or V) tile, rows of D bytes
  static constexpr uint32_t kLayout = D == 128 ? kLayoutSw128 : kLayoutSw64;
  static constexpr int kAtom = 8 * D;                  // bytes of 8 rows, the swizzle's period
  static constexpr int kQPiece = N * D;                // q_hi, then q_lo
  static constexpr int kQBytes = 2 * kQPiece;
  static constexpr int kPCols = 2 * N;                 // P^T columns: N hi, then N mid
  static constexpr int kPBytes = kTileTokens * kPCols;
  static constexpr int kPKGroup = (kPCols / 16) * 128;  // P^T stride between 8-token groups
  static constexpr int kSB = 4;                         // S^T buffers
  static constexpr int kOffK = 0;
  static constexpr int kOffV = NS * kKVBytes;
  static constexpr int kOffQ = 2 * NS * kKVBytes;
  static constexpr int kOffP = kOffQ + kQB * kQBytes;
  static constexpr int kOffSmall = kOffP + 2 * kPBytes;
  static constexpr int kSchedScratch = kOffSmall - kOffQ;  // bytes free at kernel start
  struct Small {
    uint64_t full_k[NS], empty_k[NS], full_v[NS], empty_v[NS];
    uint64_t s_full[kSB], s_free[kSB], p_full[2], o_full[2], stat_free[2];
    uint64_t m_full[2];     // [tile parity]: the tile's running references are published and
                            // those of the tile before it read
    uint64_t unit_done[2];  // [O buffer]: a unit's last P.V completed
    uint64_t o_free[2];     // [O buffer]: the unit's O is read out
    uint64_t q_full[kQB], q_empty[kQB], drain[2];
    uint32_t tmem_base;
    int abort_any;
    __align__(16) float wmax[2][2][4][N];  // [softmax warpgroup][tile parity][warp][row]
    __align__(16) float wsum[2][4][N];     // [buffer][warp][row]: per-warp sums
    float mnew[2][N];                      // [buffer][row]: the reference after the tile
    __align__(16) float mw[2][4][N];       // [softmax warpgroup][warp][row]: the warp's copy of it
    __align__(16) float aw[2][4][N];       // ... and of the factor
    float scl[2][N];                       // [buffer][row]: factor O and l take before it
    float mrun[2][N];                      // [tile parity][row]: mnew for the next tile
    __align__(16) float rowf[kQB][N];      // [Q buffer][row]: c 2^-k
    float fin_m[N], fin_l[N];              // each row's (m, l) for the direct final write
    int sched_list[kSchedMaxMine];
    int sched_meta[kSchedMaxMine][3];
    int sched_hist[kSchedHist], sched_start[kSchedBuckets];
    int sched_count;
    __align__(16) int lim[2][N];           // [softmax warpgroup][row]: key limit
    int tab[2][2][kSplitTokens / 16];      // [producer][unit parity]: block-table entries
    uint8_t sctab[2][2][kSplitTokens / 16];  // [unit parity][K, V]: the entries' scale bytes
    uint8_t sc[NS][2][8];                  // [stage][K, V][box]: scale bytes of the stage's tile
  };
  static constexpr int kSmemBytes = kOffSmall + static_cast<int>(sizeof(Small)) + 1024;
  // TMEM: S^T (N columns) x kSB buffers, then O^T (hi and mid, 2N columns) x 2
  // buffers (alternate units)
  static constexpr int kTmemCols = N == 16 ? 128 : 512;
  static constexpr uint32_t kColO = kSB * N;
};

// A scale byte, held to the range that the arithmetic covers (a byte outside
// it is reported).
__device__ __forceinline__ int checked_scale(int byte, int32_t *err) {
  if (byte < kScaleByteMin || byte > kScaleByteMax) {
    if (err) atomicOr(err, kErrScale);
    byte = byte < kScaleByteMin ? kScaleByteMin : kScaleByteMax;
  }
  return byte;
}

// A unit's block-table entries and their scale bytes on the way to shared
// memory, a lane's share in registers: the loads of the next unit go out
// before the tiles of this one are issued and are used after them.  (Under a
// saturated memory system a load takes microseconds, and at a unit's boundary
// every tile behind it waits: loading there cost 10 us per unit.)
constexpr int kTabBatch = kSplitTokens / 16 / 32;  // entries per lane at most

struct TabRegs {
  int blk[kTabBatch], kb[kTabBatch], vb[kTabBatch];
};

__device__ __forceinline__ int tab_entries(const Q8Params &p, const Unit &x) {
  const int ntok = min(kSplitTokens, x.lim_max - x.tok0);
  return (ntok + (1 << p.block_shift) - 1) >> p.block_shift;
}

__device__ __forceinline__ void load_tab(const Q8Params &p, const Unit &x, TabRegs &r, int lane) {
  const int nent = tab_entries(p, x), first = x.tok0 >> p.block_shift;
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i) {
    const int e = lane + 32 * i;
    r.blk[i] = kPastWidth;
    if (e < nent && first + e < p.max_blocks_per_seq)
      r.blk[i] = __ldg(p.block_table + x.b * p.bt_stride + first + e);
  }
}

__device__ __forceinline__ void load_scales(const Q8Params &p, const Unit &x, TabRegs &r) {
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i) {
    const int64_t blk = r.blk[i];
    r.kb[i] = r.vb[i] = 127;
    if (blk >= 0 && blk < p.num_blocks) {  // (kPastWidth is negative)
      r.kb[i] = __ldg(p.k_sc + blk * p.ksc_sb + x.kvh * p.ksc_sh);
      r.vb[i] = __ldg(p.v_sc + blk * p.vsc_sb + x.kvh * p.vsc_sh);
    }
  }
}

__device__ __forceinline__ void put_tab(const Q8Params &p, const Unit &x, const TabRegs &r, int *tab,
                                        int lane) {
  const int nent = tab_entries(p, x);
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i)
    if (lane + 32 * i < nent) tab[lane + 32 * i] = r.blk[i];
}

__device__ __forceinline__ void put_scales(const Q8Params &p, const Unit &x, const TabRegs &r,
                                           uint8_t (*sctab)[kSplitTokens / 16], int lane) {
  const int nent = tab_entries(p, x);
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i) {
    const int e = lane + 32 * i;
    if (e < nent) {
      sctab[0][e] = static_cast<uint8_t>(checked_scale(r.kb[i], p.err));
      sctab[1][e] = static_cast<uint8_t>(checked_scale(r.vb[i], p.err));
    }
  }
}

// Offset of 16-byte chunk c of row r in a K-major operand of D-byte rows under
// the tile's swizzle.
template <int D>
__device__ __forceinline__ int swz16(int r, int c) {
  return r * D + ((D == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) << 4);
}

// The query rows of unit x as q_hi and q_lo (the B operands of S^T) and their
// factors c 2^-k.  D / 8 lanes share a row, eight elements each; a pass of the
// warp takes 256 / D rows.  Rows past x.rows keep whatever the buffer holds:
// their columns of S^T are never used.
template <int D>
__device__ __forceinline__ uint4 load_q_pass(const Q8Params &p, const Unit &x, int pass, int lane) {
  constexpr int kLanes = D / 8;
  const int c = pass * (32 / kLanes) + lane / kLanes;
  if (c >= x.rows) return make_uint4(0u, 0u, 0u, 0u);
  const int r = x.row0 + c;
  const int i = r / p.G, g = r - i * p.G;
  return __ldg(reinterpret_cast<const uint4 *>(p.q + q_tok_off(p, x, i) +
                                               static_cast<int64_t>(x.kvh * p.G + g) * p.q_sh) +
               lane % kLanes);
}

template <int D, int N>
__device__ __forceinline__ void put_q_pass(const Q8Params &p, uint4 v, int pass, uint8_t *qdst,
                                           float *rowf, int lane) {
  constexpr int kLanes = D / 8;
  const int ch = lane % kLanes, c = pass * (32 / kLanes) + lane / kLanes;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;  // largest magnitude as bits: ordered like the values, NaN and inf on top
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const bool finite = top < 0x7F80u;
  // largest magnitude to [128, 256): exponent field + k = 127 + 7; held to
  // [-60, 60] so that c 2^-k 2^ek stays a normal number (rows below 2^-53
  // keep fewer bits, values past 2^68 saturate)
  int k = 134 - max(static_cast<int>(top >> 7), 1);
  k = !finite || top == 0 ? 0 : max(-60, min(60, k));
  // a row with an infinity or NaN: those elements become NaN, the rest zero
  const float f = finite ? __int_as_float((127 + k) << 23) : 0.f;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Split2 s = split_q(__fmul_rn(__uint_as_float(w[e] << 16), f),
                             __fmul_rn(__uint_as_float(w[e] & 0xFFFF0000u), f));
    hi[e] = s.hi;
    lo[e] = s.lo;
  }
  uint8_t *dst = qdst + swz16<D>(c, ch >> 1) + (ch & 1) * 8;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
  *reinterpret_cast<uint2 *>(dst + N * D) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  if (ch == 0) rowf[c] = __fmul_rn(p.cscale, __int_as_float((127 - k) << 23));
}

// One producer warp (K and the query rows, or V and the scales); the stage
// ring, the bounded waits and the exit are attn_split.cuh's produce().
template <class C>
__device__ __forceinline__ void produce_q8(const Q8Params &p, const CUtensorMap *map, uint8_t *smem,
                                           typename C::Small *sm, uint64_t *full, uint64_t *empty,
                                           int (*tabs)[kSplitTokens / 16], uint32_t dst_off,
                                           bool is_k, int lane, volatile int *abort_any,
                                           const Sched &sc) {
  constexpr int D = C::kD, N = C::kN, NS = C::kNS, QB = C::kQB;
  if (lane == 0) tma_prefetch_desc(map);
  int last_gi[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) last_gi[i] = -1;
  bool failed = false;
  Unit cur;
  int cu = next_unit<N>(p, sc, 0, cur);
  if (cu >= 0) {
    const int bmask = (1 << p.block_shift) - 1;
    int ui = 0, gi = 0;
    constexpr int kPasses = N * D / 256;
    constexpr bool kEarly = kPasses <= 8;  // the next unit's Q waits in registers too
    TabRegs tr;
    uint4 qr[kEarly ? kPasses : 1];
    auto load_q = [&](const Unit &u) {
      if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          if (i * (256 / D) < u.rows) qr[i] = load_q_pass<D>(p, u, i, lane);
      }
    };
    auto put_q = [&](const Unit &u, int ord) {
      uint8_t *dst = smem + C::kOffQ + (ord % QB) * C::kQBytes;
      float *rowf = sm->rowf[ord % QB];
      if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
          if (i * (256 / D) < u.rows) put_q_pass<D, N>(p, qr[i], i, dst, rowf, lane);
      } else {
#pragma unroll 4
        for (int i = 0; i < kPasses; ++i)
          if (i * (256 / D) < u.rows)
            put_q_pass<D, N>(p, load_q_pass<D>(p, u, i, lane), i, dst, rowf, lane);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_full[ord % QB]);
    };
    load_tab(p, cur, tr, lane);
    if (is_k) load_q(cur);
    put_tab(p, cur, tr, tabs[0], lane);
    if (is_k) {
      put_q(cur, 0);
    } else {
      load_scales(p, cur, tr);
      put_scales(p, cur, tr, sm->sctab[0], lane);
    }
    __syncwarp();
    while (true) {
      Unit nxt;
      const int nu = next_unit<N>(p, sc, cu + 1, nxt);
      if (nu >= 0) {
        load_tab(p, nxt, tr, lane);
        if (is_k) load_q(nxt);
      }
      // V: the entries have arrived a few tiles on, and their scales are
      // fetched behind the remaining ones
      const int j_scales = min(cur.n_tiles - 1, 4);
      const int *tab = tabs[ui & 1];
      for (int j = 0; j < cur.n_tiles && !failed; ++j, ++gi) {
        const int st = gi % NS;
        bool okw = true;
        if (lane == 0) okw = mbar_wait(&empty[st], ((gi / NS) & 1) ^ 1, abort_any, p.wait_ns);
        if (!__shfl_sync(0xffffffffu, okw ? 1 : 0, 0)) {
          failed = true;
          break;
        }
        const int tok0 = cur.tok0 + j * kTileTokens;
        const int nvalid = min(kTileTokens, cur.lim_max - tok0);
        const int nbox = (nvalid + p.box_slots - 1) >> p.box_shift;
        int errs = 0;
        if (lane < nbox) {
          const int tok = tok0 + (lane << p.box_shift);
          const int e = (tok - cur.tok0) >> p.block_shift;
          const int blk = tab[e];
          if (blk == kPastWidth) {
            errs = kErrTableWidth;
          } else if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks) {
            errs = kErrBadBlock;
          } else {
            uint8_t *d0 = smem + dst_off + st * C::kKVBytes + (lane << p.box_shift) * D;
            const int slot = tok & bmask;
            const int c1 = p.map_head_first ? cur.kvh : slot;
            const int c2 = p.map_head_first ? slot : cur.kvh;
            mbar_expect_tx(&full[st], static_cast<uint32_t>(p.box_slots * D));
            tma_load_4d(d0, map, &full[st], 0, c1, c2, blk);
          }
          if (!is_k) {
            sm->sc[st][0][lane] = sm->sctab[ui & 1][0][e];
            sm->sc[st][1][lane] = sm->sctab[ui & 1][1][e];
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[st]);
          last_gi[st] = gi;
        }
        if (errs && p.err) atomicOr(p.err, errs);
        if (!is_k && nu >= 0 && j == j_scales) load_scales(p, nxt, tr);
      }
      if (failed || nu < 0) break;
      // (the other parity's entries were last read for the unit before this one)
      put_tab(p, nxt, tr, tabs[(ui + 1) & 1], lane);
      if (!is_k) put_scales(p, nxt, tr, sm->sctab[(ui + 1) & 1], lane);
      // The next unit's Q goes into the buffer of the unit before this one,
      // once its last QK^T and its epilogue (staged there) are done; see
      // produce() for why the wait comes after this unit's last tile.
      if (is_k) {
        const int qb = (ui + 1) % QB;
        bool okq = true;
        if (lane == 0) okq = mbar_wait(&sm->q_empty[qb], (((ui + 1) / QB) & 1) ^ 1, abort_any, p.wait_ns);
        if (!__shfl_sync(0xffffffffu, okq ? 1 : 0, 0)) {
          failed = true;
          break;
        }
        put_q(nxt, ui + 1);
      }
      __syncwarp();
      ++ui;
      cur = nxt;
      cu = nu;
    }
  }
  if (lane == 0) {
    // every copy this warp issued lands before the CTA exits (bounded)
    volatile int no_abort = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (last_gi[i] >= 0) mbar_wait(&full[i], (last_gi[i] / NS) & 1, &no_abort);
  }
}

template <int D, int N, int NS>
__global__ void __launch_bounds__(kQ8Threads, 1)
    attn_split_q8_kernel(const __grid_constant__ Q8Params p,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v) {
  using C = Q8Cfg<D, N, NS>;
  constexpr int QB = C::kQB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto *sm = reinterpret_cast<typename C::Small *>(smem + C::kOffSmall);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int *abort_any = &sm->abort_any;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full_k[i], 1);
      mbar_init(&sm->empty_k[i], 1);
      mbar_init(&sm->full_v[i], 1);
      mbar_init(&sm->empty_v[i], 1);
    }
    for (int i = 0; i < C::kSB; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->s_free[i], 4);   // one arrival per warp of a softmax warpgroup
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->p_full[i], 4);   // one arrival per warp of a softmax warpgroup
      mbar_init(&sm->o_full[i], 1);
      mbar_init(&sm->stat_free[i], 4);
      mbar_init(&sm->m_full[i], 4);   // one arrival per warp of a softmax warpgroup
      mbar_init(&sm->unit_done[i], 1);
      mbar_init(&sm->o_free[i], 4);   // one arrival per correction warp
      mbar_init(&sm->q_full[i], 1);
      mbar_init(&sm->q_empty[i], 2);  // the unit's last QK^T, and its epilogue
      mbar_init(&sm->drain[i], 1);
    }
    sm->abort_any = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&sm->tmem_base, C::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm->tmem_base;
  const uint32_t sbase = smem_u32(smem);
  // the Q and P^T buffers are not in use yet: the schedule's scratch
  Sched sc = strided_sched(p);
  if (p.sched) {
    build_schedule<N>(p, smem + C::kOffQ, C::kSchedScratch, sm->sched_hist, sm->sched_start,
                      sm->sched_list, sm->sched_meta, &sm->sched_count);
    if (sm->sched_count >= 0) {
      sc = Sched{sm->sched_list, sm->sched_meta, sm->sched_count};
    } else if (sc.count <= kSchedMaxMine) {
      // nothing to balance: the stride-grid deal as a list, so that no role
      // reads global memory between units
      for (int k = threadIdx.x; k < sc.count; k += kQ8Threads) {
        const int u = sc.unit(k), b = unit_seq(p, u);
        sm->sched_list[k] = u;
        sm->sched_meta[k][0] = __ldg(p.seqlens + b);
        sm->sched_meta[k][1] = p.cu_q ? __ldg(p.cu_q + b) : 0;
        sm->sched_meta[k][2] = p.cu_q ? __ldg(p.cu_q + b + 1) : 0;
      }
      __syncthreads();
      sc = Sched{sm->sched_list, sm->sched_meta, sc.count};
    }
  }

  if (warp == kKWarp) {
    produce_q8<C>(p, &map_k, smem, sm, sm->full_k, sm->empty_k, sm->tab[0], C::kOffK, true, lane,
                  abort_any, sc);
  } else if (warp == kVWarp) {
    produce_q8<C>(p, &map_v, smem, sm, sm->full_v, sm->empty_v, sm->tab[1], C::kOffV, false, lane,
                  abort_any, sc);
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ------------------------------------------------------------------
    // MMA issuers, one thread each: QK^T of every tile as soon as its K and a
    // S^T buffer are there, and P.V of every tile as soon as its P and V are.
    // One thread for both spent 1750 cycles on a tile (issue of 12 small MMAs
    // and 5 commits, and the waits between), more than the 1500 that the
    // tile's 32 KB take from memory.
    // ------------------------------------------------------------------
    if (lane == 0) {
      const bool is_qk = warp == kMmaWarp;
      // A = K tile, B = q_hi / q_lo (K-major); A = V^T, B = P^T (MN-major)
      constexpr uint32_t kQkHi = idesc_f8(128, N, kFmtE4M3, kFmtE4M3, 0, 0);
      constexpr uint32_t kQkLo = idesc_f8(128, N, kFmtE4M3, kFmtE5M2, 0, 0);
      constexpr uint32_t kPv = idesc_f8(128, C::kPCols, kFmtE4M3, kFmtE4M3, 1, 1);
      int gi = 0, ui = 0;
      bool failed = false;
      for (int k = 0; k < sc.count && !failed; ++k) {
        const Unit x = sc.get<N>(p, k);
        if (x.n_tiles == 0) continue;
        if (is_qk) {
          const int qb = ui % QB;
          if (!mbar_wait(&sm->q_full[qb], (ui / QB) & 1, abort_any, p.wait_ns)) {
            failed = true;
            break;
          }
          const uint64_t bh = smem_desc(sbase + C::kOffQ + qb * C::kQBytes, 16, C::kAtom, C::kLayout);
          for (int j = 0; j < x.n_tiles; ++j, ++gi) {
            const int st = gi % NS, sb = gi % C::kSB;
            if (!mbar_wait(&sm->full_k[st], (gi / NS) & 1, abort_any, p.wait_ns) ||
                !mbar_wait(&sm->s_free[sb], ((gi / C::kSB) & 1) ^ 1, abort_any, p.wait_ns)) {
              failed = true;
              break;
            }
            tc_fence_after_sync();
            const uint64_t a = smem_desc(sbase + C::kOffK + st * C::kKVBytes, 16, C::kAtom, C::kLayout);
            const uint32_t d = tmem + sb * N;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              umma_f8(d, a + kk * 2, bh + kk * 2, kQkHi, kk > 0 ? 1u : 0u);
              umma_f8(d, a + kk * 2, bh + (C::kQPiece >> 4) + kk * 2, kQkLo, 1u);
            }
            umma_commit(&sm->s_full[sb]);
            umma_commit(&sm->empty_k[st]);
            if (j == x.n_tiles - 1) umma_commit(&sm->q_empty[qb]);
          }
        } else {
          const int ob = ui & 1;
          const uint32_t d = tmem + C::kColO + ob * C::kPCols;
          if (!mbar_wait(&sm->o_free[ob], ((ui >> 1) & 1) ^ 1, abort_any, p.wait_ns)) {
            failed = true;
            break;
          }
          for (int j = 0; j < x.n_tiles; ++j, ++gi) {
            const int st = gi % NS, bb = gi & 1;
            if (!mbar_wait(&sm->full_v[st], (gi / NS) & 1, abort_any, p.wait_ns) ||
                !mbar_wait(&sm->p_full[bb], (gi >> 1) & 1, abort_any, p.wait_ns)) {
              failed = true;
              break;
            }
            tc_fence_after_sync();
            // V^T: MN-major, 32 tokens (four 8-token atoms) per step.  D = 64:
            // both M halves read the same 64 columns; lanes 64..127 are unused.
            const uint64_t a = smem_desc(sbase + C::kOffV + st * C::kKVBytes, 0, C::kAtom, C::kLayout);
            // P^T: MN-major, no swizzle; 16-column groups 128 B apart, 8-token
            // groups kPKGroup apart
            const uint64_t b = smem_desc(sbase + C::kOffP + bb * C::kPBytes, C::kPKGroup, 128,
                                         kLayoutInterleave);
#pragma unroll
            for (int kk = 0; kk < kTileTokens / 32; ++kk)
              umma_f8(d, a + kk * (4 * C::kAtom >> 4), b + kk * (4 * C::kPKGroup >> 4), kPv,
                      (j == 0 && kk == 0) ? 0u : 1u);
            umma_commit(&sm->o_full[bb]);
            umma_commit(&sm->empty_v[st]);
            if (j == x.n_tiles - 1) umma_commit(&sm->unit_done[ob]);
          }
        }
        ++ui;
      }
      // every MMA this thread issued completes before TMEM is released
      (void)failed;
      uint64_t *drain = &sm->drain[is_qk ? 0 : 1];
      umma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
  } else if (warp < kCorrWarp0) {
    // ------------------------------------------------------------------
    // Softmax warpgroups: warpgroup wg takes the tiles with gi % 2 == wg;
    // thread t <-> TMEM lane t <-> token t of the tile.
    // ------------------------------------------------------------------
    const int wg = warp >> 2, wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t bar_id = 1 + wg;
    const float NEG_INF = neg_inf();
    int gbase = 0, uo = 0;  // uo: ordinal of the unit among this CTA's units with work
    bool stop = false;
    for (int k = 0; k < sc.count && !stop; ++k) {
      const Unit x = sc.get<N>(p, k);
      if (x.n_tiles == 0) continue;
      const uint32_t ocol = tmem + lane_off + C::kColO + (uo & 1) * C::kPCols;  // this unit's O^T
      if (t < N) {
        int lim = 0;
        if (t < x.rows) {
          const int i = (x.row0 + t) / p.G;
          lim = x.seqlen;
          if (p.causal) lim = min(lim, x.seqlen - x.nq + i + 1);
          lim = lim > 0 ? lim : 0;
        }
        sm->lim[wg][t] = lim;
      }
      // the unit's Q and row factors are staged (the buffer is not filled
      // again before this unit's epilogue, so the phase cannot move on)
      const bool okq = mbar_wait(&sm->q_full[uo % QB], (uo / QB) & 1, abort_any, p.wait_ns);
      const float *rowf = sm->rowf[uo % QB];
      if (wg_bar_or(bar_id, !okq)) {
        stop = true;
        break;
      }
      for (int j = 0; j < x.n_tiles; ++j) {
        const int gi = gbase + j;
        if ((gi & 1) != wg) continue;
        const int bb = wg, st = gi % NS, sb = gi % C::kSB, par = (gi >> 1) & 1;
        // V landed: the stage's scale bytes are staged with it (the stage is
        // not refilled before this tile's P.V)
        bool ok = mbar_wait(&sm->full_v[st], (gi / NS) & 1, abort_any, p.wait_ns);
        ok = mbar_wait(&sm->s_full[sb], (gi / C::kSB) & 1, abort_any, p.wait_ns) && ok;
        // P^T[bb] is free once P.V of tile gi - 2 is done, the row statistics
        // once the correction of tile gi - 2 has read them
        ok = mbar_wait(&sm->o_full[bb], par ^ 1, abort_any, p.wait_ns) && ok;
        ok = mbar_wait(&sm->stat_free[bb], par ^ 1, abort_any, p.wait_ns) && ok;
        tc_fence_after_sync();
        float sv[N];
#pragma unroll
        for (int ch = 0; ch < N / 16; ++ch)
          if (ch * 16 < x.rows)
            tmem_ld16(tmem + lane_off + sb * N + ch * 16, *reinterpret_cast<float(*)[16]>(&sv[ch * 16]));
        const int tok0 = x.tok0 + j * kTileTokens;
        const int tok = tok0 + t;
        const bool held = tok < x.lim_max;
        const int kb = held ? sm->sc[st][0][t >> p.box_shift] : 127;
        const int vb = held ? sm->sc[st][1][t >> p.box_shift] : 127;
        const float ks = scale_of(kb), ev = static_cast<float>(vb - 127), iv = inv_scale_of(vb);
#pragma unroll
        for (int ch = 0; ch < N / 16; ++ch)
          if (ch * 16 < x.rows) tmem_ld_wait_for(*reinterpret_cast<float(*)[16]>(&sv[ch * 16]));
        // the S^T buffer is read
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->s_free[sb]);
        if (tok0 + kTileTokens > x.lim_max && ok && !held) {
          // The last tile: keys past the loaded range hold stale bytes; zero
          // those V rows so that 0 * V stays 0 in P.V.
          uint4 *vrow = reinterpret_cast<uint4 *>(smem + C::kOffV + st * C::kKVBytes + t * D);
#pragma unroll
          for (int k16 = 0; k16 < D / 16; ++k16) vrow[k16] = make_uint4(0u, 0u, 0u, 0u);
        }
        float(*wmax)[N] = sm->wmax[wg][par];
#pragma unroll
        for (int q4 = 0; q4 < N / 4; ++q4) {
          if (q4 * 4 < x.rows) {  // warp-uniform: padded rows need no reduction
            const int4 lim = *reinterpret_cast<const int4 *>(&sm->lim[wg][4 * q4]);
            const float4 rf = *reinterpret_cast<const float4 *>(&rowf[4 * q4]);
            const int lims[4] = {lim.x, lim.y, lim.z, lim.w};
            const float rfs[4] = {rf.x, rf.y, rf.z, rf.w};
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = 4 * q4 + e;
              // (masked, and rows past x.rows, whose limit is 0: the score
              // itself is -inf from here on)
              const bool seen = tok < lims[e];
              sv[c] = seen ? sv[c] : NEG_INF;
              v[e] = seen ? __fmaf_rn(sv[c], __fmul_rn(rfs[e], ks), ev) : NEG_INF;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = warp_max(v[e]);
            if (lane == 0)
              *reinterpret_cast<float4 *>(&wmax[wq][4 * q4]) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
        // the running references: the previous tile's, this tile's.  Every
        // warp works them out for itself (lane = row), so that the chain from
        // tile to tile has no barrier in it; warp 0 publishes them.
        if (gi > 0)
          ok = mbar_wait(&sm->m_full[(gi - 1) & 1], ((gi - 1) >> 1) & 1, abort_any, p.wait_ns) && ok;
        bool moved = false;
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 32) {
          const int c = c0 + lane;
          if (c < N) {
            float m_new = NEG_INF, a = 1.f;
            if (c < x.rows) {
              const float tmax = fmaxf(fmaxf(wmax[0][c], wmax[1][c]), fmaxf(wmax[2][c], wmax[3][c]));
              const float m_prev = j > 0 ? sm->mrun[(gi - 1) & 1][c] : NEG_INF;
              m_new = (tmax > __fadd_rn(m_prev, kRefTop)) ? __fsub_rn(tmax, kRefDrop) : m_prev;
              a = (m_prev == NEG_INF || m_new == m_prev) ? 1.f : ex2(__fsub_rn(m_prev, m_new));
            }
            sm->mw[wg][wq][c] = m_new;
            sm->aw[wg][wq][c] = a;
            moved = moved || a != 1.f;
            if (wq == 0) {
              sm->mrun[gi & 1][c] = m_new;
              sm->mnew[bb][c] = m_new;
              sm->scl[bb][c] = a;
            }
          }
        }
        const bool resc = __any_sync(0xffffffffu, moved);  // (also orders mw / aw for the warp)
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->m_full[gi & 1]);
        if (resc) {
          // O^T holds the unit's tiles < gi once P.V(gi - 1) is done (see
          // attn_split.cuh on the parity)
          ok = mbar_wait(&sm->o_full[(gi - 1) & 1], ((gi - 1) >> 1) & 1, abort_any, p.wait_ns) && ok;
          if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after_sync();
#pragma unroll
            for (int ch = 0; ch < N / 16; ++ch) {
              if (ch * 16 < x.rows) {  // warp-uniform
                float hi[16], mid[16];
                tmem_ld16(ocol + ch * 16, hi);
                tmem_ld16(ocol + N + ch * 16, mid);
                tmem_ld_wait_for(hi);
                tmem_ld_wait_for(mid);
                uint32_t wh[16], wm[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float a = sm->aw[wg][wq][ch * 16 + e];
                  wh[e] = __float_as_uint(__fmul_rn(hi[e], a));
                  wm[e] = __float_as_uint(__fmul_rn(mid[e], a));
                }
                tmem_st16(ocol + ch * 16, wh);
                tmem_st16(ocol + N + ch * 16, wm);
              }
            }
            tmem_st_wait();
          }
        }
        // P^T row t: one 16-byte chunk of hi and of mid per 16 rows
        uint8_t *prow = smem + C::kOffP + bb * C::kPBytes + (t >> 3) * C::kPKGroup + (t & 7) * 16;
#pragma unroll
        for (int grp = 0; grp < N / 16; ++grp) {
          uint32_t wh[4], wm[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c0 = grp * 16 + 4 * e;
            SplitP a{0u, 0u}, b{0u, 0u};
            if (c0 < x.rows) {  // groups of padded rows keep p = 0
              const float4 rf = *reinterpret_cast<const float4 *>(&rowf[c0]);
              const float4 mm = *reinterpret_cast<const float4 *>(&sm->mw[wg][wq][c0]);
              const float rfs[4] = {rf.x, rf.y, rf.z, rf.w}, ms[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sv[c0 + i] = (sv[c0 + i] == NEG_INF)
                                 ? 0.f
                                 : ex2(__fmaf_rn(sv[c0 + i], __fmul_rn(rfs[i], ks), __fsub_rn(ev, ms[i])));
              a = split_p(sv[c0], sv[c0 + 1]);
              b = split_p(sv[c0 + 2], sv[c0 + 3]);
            }
            wh[e] = a.hi | (b.hi << 16);
            wm[e] = a.mid | (b.mid << 16);
          }
          *reinterpret_cast<uint4 *>(prow + grp * 128) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
          *reinterpret_cast<uint4 *>(prow + (N / 16 + grp) * 128) = make_uint4(wm[0], wm[1], wm[2], wm[3]);
        }
#pragma unroll
        for (int q4 = 0; q4 < N / 4; ++q4) {
          if (q4 * 4 < x.rows) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(sv[4 * q4 + e], iv);
            warp_sum4_lane0(v);
            if (lane == 0)
              *reinterpret_cast<float4 *>(&sm->wsum[bb][wq][4 * q4]) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full[bb]);
      }
      gbase += x.n_tiles;
      ++uo;
    }
    (void)stop;
  } else if (warp < kCorrWarp0 + 4) {
    // ------------------------------------------------------------------
    // Correction + epilogue warpgroup: thread r (< rows) owns row r's
    // running l; at the unit's end thread t <-> column d of O^T.
    // ------------------------------------------------------------------
    const int wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    constexpr uint32_t bar_id = 3;
    const float NEG_INF = neg_inf();
    float acc[N];
    float m_run = NEG_INF, l_run = 0.f;
    int gbase = 0, cui = 0;
    bool bulk_out = false;   // thread 0 has bulk stores to complete before exit
    bool stop = false;
    for (int k = 0; k < sc.count && !stop; ++k) {
      const Unit x = sc.get<N>(p, k);
      if (t == 0) check_sequence(p, x);
      if (x.n_tiles == 0) {
        // direct write: rows of this unit see no key (out = 0, lse = -inf)
        if (p.direct && x.rows > 0) {
#pragma unroll
          for (int c = 0; c < N; ++c) acc[c] = 0.f;
          float none[N];
#pragma unroll
          for (int c = 0; c < N; ++c) none[c] = NEG_INF;
          write_final_cols<D, N>(p, x, t, acc, none, none);
        }
        continue;
      }
      m_run = NEG_INF;
      l_run = 0.f;
      for (int j = 0; j < x.n_tiles; ++j) {
        const int gi = gbase + j, bb = gi & 1, par = (gi >> 1) & 1;
        const bool ok = mbar_wait(&sm->p_full[bb], par, abort_any, p.wait_ns);  // the tile's row statistics
        if (t < x.rows) {
          const float lt = __fadd_rn(__fadd_rn(sm->wsum[bb][0][t], sm->wsum[bb][1][t]),
                                     __fadd_rn(sm->wsum[bb][2][t], sm->wsum[bb][3][t]));
          l_run = __fmaf_rn(l_run, sm->scl[bb][t], lt);
          m_run = sm->mnew[bb][t];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->stat_free[bb]);  // the tile's statistics are read
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
      }
      if (stop) break;
      {
        const int ob = cui & 1;
        const bool ok = mbar_wait(&sm->unit_done[ob], (cui >> 1) & 1, abort_any, p.wait_ns);
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int ch = 0; ch < N / 16; ++ch) {
          if (ch * 16 < x.rows) {  // warp-uniform
            float hi[16], mid[16];
            tmem_ld16(tmem + lane_off + C::kColO + ob * C::kPCols + ch * 16, hi);
            tmem_ld16(tmem + lane_off + C::kColO + ob * C::kPCols + N + ch * 16, mid);
            tmem_ld_wait_for(hi);
            tmem_ld_wait_for(mid);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[ch * 16 + e] = __fmaf_rn(mid[e], kMidScale, hi[e]);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->o_free[ob]);
      }
      uint8_t *qstage = smem + C::kOffQ + (cui % QB) * C::kQBytes;  // this unit's Q: its QK^T are done
      if (p.direct) {
        // every row of the call has at most one split: out / lse here
        if (t < x.rows) {
          sm->fin_m[t] = m_run;
          sm->fin_l[t] = l_run;
        }
        wg_bar_or(bar_id, false);
        if (p.out_vec) {
          // out rows through the unit's Q buffer and bulk stores
          static_assert(C::kQBytes >= N * D * 2, "the out rows of a unit fit its Q buffer");
          __nv_bfloat16 *stage = reinterpret_cast<__nv_bfloat16 *>(qstage);
          write_final_cols<D, N>(p, x, t, acc, sm->fin_m, sm->fin_l, stage);
          fence_proxy_async_smem();
          wg_bar_or(bar_id, false);
          if (t == 0) {
            for (int c = 0; c < x.rows; ++c) {
              const int r = x.row0 + c;
              const int i = r / p.G, g = r - i * p.G;
              bulk_store(p.out + o_tok_off(p, x, i) + (x.kvh * p.G + g) * p.o_sh, stage + c * D,
                         D * 2);
            }
            bulk_commit();
            bulk_out = true;
          }
        } else {
          write_final_cols<D, N>(p, x, t, acc, sm->fin_m, sm->fin_l);
        }
      } else {
        // unnormalised split partial of every real row, through the Q buffer
        const int64_t S = p.n_splits;
        float *stage = reinterpret_cast<float *>(qstage);
        constexpr int kRowsStaged = C::kQBytes / (D * 4);
        for (int c0 = 0; c0 < x.rows; c0 += kRowsStaged) {
          if (c0 > 0 && t == 0) bulk_wait_read<0>();  // the previous round has read the stage
          if (c0 > 0) wg_bar_or(bar_id, false);
#pragma unroll
          for (int c = 0; c < N; ++c)
            if (c >= c0 && c < min(x.rows, c0 + kRowsStaged) && t < D)
              stage[(c - c0) * D + t] = acc[c];
          fence_proxy_async_smem();
          wg_bar_or(bar_id, false);
          if (t == 0) {
            for (int c = c0; c < min(x.rows, c0 + kRowsStaged); ++c) {
              const int r = x.row0 + c;
              const int i = r / p.G, g = r - i * p.G;
              const int64_t row_id = (x.q0 + i) * p.Hq + x.kvh * p.G + g;
              bulk_store(p.ws_acc + (row_id * S + x.s) * D, stage + (c - c0) * D, D * 4);
            }
            bulk_commit();
            bulk_out = true;
          }
        }
        if (t < x.rows) {
          const int r = x.row0 + t;
          const int i = r / p.G, g = r - i * p.G;
          const int64_t row_id = (x.q0 + i) * p.Hq + x.kvh * p.G + g;
          *reinterpret_cast<float2 *>(p.ws_ml + (row_id * S + x.s) * 2) = make_float2(m_run, l_run);
        }
      }
      // the stage has been read: the producer may load a later unit's Q here
      if (t == 0) {
        if (bulk_out) bulk_wait_read<0>();
        mbar_arrive(&sm->q_empty[cui % QB]);
      }
      ++cui;
      gbase += x.n_tiles;
    }
    // the partials are complete in global memory before the CTA leaves
    if (bulk_out) bulk_wait<0>();
    (void)stop;
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && sm->abort_any && p.err) atomicOr(p.err, kErrTimeout);
}

}  // namespace pkv
