// attn_split_q8.cuh -- split-KV attention over an 8-bit paged cache, few query
// rows per KV head (decode, multi-token decode), sm_100a.
//
// The cache holds K and V as e4m3 values with a scale 2^e for each block of
// tokens and KV head (f8.cuh).  Units, splits, tiles, schedule, roles and the
// merge are those of attn_split.cuh; what differs is the arithmetic of a tile,
// which runs on the 8-bit tensor-core path without ever widening the cache:
//   S^T   = K8 * [q_hi | q_lo]^T   (kind::f8f6f4, M = 128 tokens), the query
//           row taken apart exactly into two 8-bit operands side by side
//           (split_q) and S = S_hi + S_lo / 16, q . k8 to fp32 accumulation;
//   w     = S * (c 2^-k 2^ek) + ev, per token: ek and ev are the exponents of
//           its K and V scales, k the query row's, c = softmax scale * log2 e.
//           w is the base-2 score plus the log of the V scale, so 2^w weighs
//           the token's 8-bit V directly;
//   (two tiles at a time from here on, 256 tokens, a thread holding a token of
//   each: the chain of reductions, barriers and fences is latency, and its
//   length hardly depends on how much it carries)
//   m     the row's running reference (-inf at the split's start) rises to
//           max(w) - kRefDrop when max(w) > m + kRefTop; P = 2^(w - m) is then
//           at most 2^kRefTop and at least 2^kRefDrop for the largest token;
//   O^T  += V8^T * [P_hi | P_mid | P_lo]^T, P as three 8-bit operands side by
//           side (split_p), joined (join_p) at the split's end;
//   l     = sum of e = 2^(w - ev - m) over the tokens, in fp32, and P = e 2^ev
//           from it.  (The other way round, e = P 2^-ev, P is flushed to zero
//           beside a scale 2^126 times its own, as a block of zeros may have,
//           and the token drops out of the sum.  e is at least 2^(kRefDrop - 63)
//           for the largest token, so what is flushed of it does not count.
//           For the same reason a move of m scales l in two steps, and the
//           merge's fold does: l may be 2^90, and the factor below 2^-126.)
// (m, l, O) is a partial in the form the merge folds: out = O / l and lse =
// (m + log2 l) ln 2.  Folding the V scale into the exponent keeps every
// operand of one MMA on one scale, whatever the blocks' scales are, and lets
// the reference follow what the tokens contribute to the output.
//
// What bounds it: the cache bytes, and how fast the TMA unit takes boxes.  A
// 128-token tile of one KV head is 32 KB (head_dim 128) against 64 KB for bf16,
// so the softmax chain has half the time per tile; with 8-bit operands read in
// place the tensor cores and the shared memory see no conversion traffic
// (widening the tile to bf16 in shared memory would move 5 bytes per cache byte
// through it).  4 x 131072 tokens in 16-token blocks, 4 rows per KV head: 197
// to 199.5 us from device to device, 5.4 TB/s (the loads alone: 188, a box of 16
// rows at a time); 64 contexts up to 32768 in 256-token blocks: 185 us, 5.57
// TB/s.  With more rows per unit the latency of the softmax takes over -- two
// warpgroups that pass the reference on from pair to pair, a thread's scores
// past its registers (64 bytes spilled for 8 rows, 212 for 16) -- and no unit of
// the SM is full: 64 x 16384 tokens with 8 rows per KV head 221 us, 4.9 TB/s,
// with 16 rows 379 us, 2.8 TB/s (7400 cycles a pair of tiles; still ahead of the
// row-major kernel's 1.7 TB/s at 16 rows).
#pragma once

#include "attn_split.cuh"
#include "f8.cuh"

namespace pkv {

// P <= 2^15 fits fp16 and e5m2 with room for the pieces' factors; the reference
// moves when the largest token passes it, and then to 2^kRefDrop below that
// token, so a row's largest P stays in [2^kRefDrop, 2^kRefTop] and the rounding
// of the smallest, 2^-25, is at most 2^-34 of it: less than fp32's own over a
// split's 4096 tokens.  Each move waits for the P.V under way and rescales O,
// 6000 cycles without a new tile: with a distance of 2 between the two, moves
// in the first tiles of every split cost a third of the time.
constexpr float kRefTop = 15.f, kRefDrop = 9.f;

struct Q8Params : AttnParams {
  const uint8_t *k_sc, *v_sc;  // scale bytes of (block, KV head)
  int64_t ksc_sb, ksc_sh, vsc_sb, vsc_sh;
  int box_shift;               // log2(box_slots)
};

// Roles: NW softmax warpgroups that take the pairs of tiles in turn, the
// correction + epilogue warpgroup, a warp for what a unit needs (table, scales,
// Q), kLoaders warps for K and V, one each for QK^T (+ TMEM owner) and P.V.
// N: rows that a unit can hold, 4, 8 or 16 -- the smallest that holds the call's
// (everything per row is unrolled over it: with 16 throughout, 4 rows ran 900
// instructions of which they needed a third, past the instruction cache).
template <int D, int N, int NSK, int NSV>
struct Q8Cfg {
  static_assert(D == 64 || D == 128, "head_dim 64 or 128");
  static_assert(N == 4 || N == 8 || N == 16, "rows per unit");
  static constexpr int kD = D, kN = N, kQB = 2;
  static constexpr int kNW = 2;
  static constexpr int kNP = 2;                // P^T buffers (a pair of tiles each)
  static constexpr int kCorr0 = 4 * kNW;       // first correction warp
  // A 16-row box takes the TMA unit 100 cycles, but one warp only gets a box
  // out every 145; with two warps each for K and V, on alternate stages, the
  // unit's queue stays full (loads alone: 3.1 TB/s for 16-token blocks with
  // one warp, 4.3 with two, 5.7 with four).
  static constexpr int kLoaders = 4;
  static constexpr int kPrepW = kCorr0 + 4, kLoadW = kCorr0 + 5, kQkW = kLoadW + kLoaders, kPvW = kQkW + 1;
  static constexpr int kWarps = kPvW + 1;
  static constexpr int kUS = 3;                // units whose table and scales are in shared memory
  static constexpr int kKVBytes = kTileTokens * D;     // one K (or V) tile, rows of D bytes
  static constexpr uint32_t kLayout = D == 128 ? kLayoutSw128 : kLayoutSw64;
  static constexpr int kAtom = 8 * D;                  // bytes of 8 rows, the swizzle's period
  static constexpr int kQCols = N == 16 ? 32 : 16;     // S^T columns: N hi, N lo (and padding)
  static constexpr int kQBytes = kQCols * D;
  static constexpr int kPCols = N == 4 ? 16 : N == 8 ? 32 : 48;  // P^T columns: N hi, mid, lo (and padding)
  static constexpr int kPTile = kTileTokens * kPCols;
  static constexpr int kPBytes = 2 * kPTile;
  static constexpr int kPKGroup = (kPCols / 16) * 128;  // P^T stride between 8-token groups
  static constexpr int kSB = 4;                         // S^T buffers
  // Scale bytes per tile.  K of tile g + kSC is issued when K of tile g + kSC -
  // NSK is used, so its S^T buffer was free: tile g + kSC - NSK - kSB's softmax
  // had read its S^T, and its scales before that.
  static constexpr int kSC = 16;
  static_assert(NSK + kSB <= kSC, "a slot of scale bytes is rewritten after its tile's softmax read it");
  static constexpr int kOffK = 0;
  static constexpr int kOffV = NSK * kKVBytes;
  static constexpr int kOffQ = (NSK + NSV) * kKVBytes;
  static constexpr int kOffP = kOffQ + kQB * kQBytes;
  static constexpr int kOffSmall = kOffP + kNP * kPBytes;
  static constexpr int kSchedScratch = kOffSmall - kOffQ;  // bytes free at kernel start
  // a unit's query rows as they are in memory
  static constexpr int kRawBytes = N * D * 2;
  struct Small {
    __align__(16) uint8_t raw_q[kRawBytes];
    uint64_t full_k[NSK], empty_k[NSK], full_v[NSV], empty_v[NSV];
    uint64_t sc_full[kSC];  // [tile % kSC]: the tile's scale bytes are staged
    uint64_t tab_full[kUS], tab_free[kUS];  // [unit % kUS]: its table and scales are there; are used
    uint64_t s_full[kSB], s_free[kSB], p_full[kNP], o_full[kNP], stat_free[kNP];
    uint64_t m_full[2];     // [pair parity]: the pair's running references are published and
                            // those of the pair before it read
    uint64_t unit_done[2];  // [O buffer]: a unit's last P.V completed
    uint64_t o_free[2];     // [O buffer]: the unit's O is read out
    uint64_t q_full[kQB], q_empty[kQB], drain[2];
    uint32_t tmem_base;
    int abort_any;
    __align__(16) float wmax[kNW][2][4][N];  // [softmax warpgroup][its pair's parity][warp][row]
    __align__(16) float wsum[kNP][4][N];   // [buffer][warp][row]: per-warp sums
    float mnew[kNP][N];                    // [buffer][row]: the reference after the pair
    __align__(16) float mw[kNW][4][N];     // [softmax warpgroup][warp][row]: the warp's copy of it
    __align__(16) float aw[kNW][4][N];     // ... and of the factor
    float scl[kNP][N];                     // [buffer][row]: root of the factor that l takes before it
    float mrun[2][N];                      // [pair parity][row]: mnew for the next pair
    __align__(16) float rowf[kQB][N];      // [Q buffer][row]: c 2^-k
    float fin_m[N], fin_l[N];              // each row's (m, l) for the direct final write
    int sched_list[kSchedMaxMine];
    int sched_meta[kSchedMaxMine][3];
    Unit units[kSchedMaxMine];             // this CTA's units, worked out once
    int sched_hist[kSchedHist];
    int sched_count;
    __align__(16) int lim[kNW][N];         // [softmax warpgroup][row]: key limit
    int tab[kUS][kSplitTokens / 16];       // [unit % kUS]: block-table entries
    uint16_t sctab[kUS][kSplitTokens / 16];  // [unit % kUS]: the entries' scale bytes, K | V << 8
    uint16_t sc[kSC][8];                   // [tile % kSC][box]: the tile's scale bytes
  };
  static constexpr int kSmemBytes = kOffSmall + static_cast<int>(sizeof(Small)) + 1024;
  // TMEM: S^T (hi and lo) x kSB buffers, then O^T (hi, mid and lo) x 2 buffers
  // (alternate units)
  static constexpr uint32_t kColO = kSB * kQCols;
  static constexpr int kTmemCols = kColO + 2 * kPCols <= 128 ? 128 : 256;
  static_assert(kColO + 2 * kPCols <= kTmemCols, "TMEM columns");
};

// C consecutive columns of the thread's TMEM lane (C a multiple of 8).
template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float *v) {
#pragma unroll
  for (int c = 0; c + 16 <= C; c += 16) tmem_ld16(taddr + c, *reinterpret_cast<float(*)[16]>(v + c));
  if constexpr (C % 16 == 8) tmem_ld8(taddr + C - 8, v + C - 8);
}
template <int C>
__device__ __forceinline__ void tmem_ld_cols_wait(float *v) {
#pragma unroll
  for (int c = 0; c + 16 <= C; c += 16) tmem_ld_wait_for(*reinterpret_cast<float(*)[16]>(v + c));
  if constexpr (C % 16 == 8) tmem_ld_wait_for8(v + C - 8);
}

// A scale byte, held to the range that the arithmetic covers (a byte outside
// it is reported).
__device__ __forceinline__ int checked_scale(int byte, int32_t *err) {
  if (byte < kScaleByteMin || byte > kScaleByteMax) {
    if (err) atomicOr(err, kErrScale);
    byte = byte < kScaleByteMin ? kScaleByteMin : kScaleByteMax;
  }
  return byte;
}

// A unit's block-table entries, their scale bytes and its query rows come from
// a warp of their own, units ahead of the tiles: under a saturated memory
// system a load takes microseconds, and in a producer warp every tile behind
// it waits (10 us per unit, a third of the time).
constexpr int kTabBatch = kSplitTokens / 16 / 32;  // entries per lane at most

__device__ __forceinline__ int tab_entries(const Q8Params &p, const Unit &x) {
  const int ntok = min(kSplitTokens, x.lim_max - x.tok0);
  return (ntok + (1 << p.block_shift) - 1) >> p.block_shift;
}

// (asynchronous: complete after cp_async_wait<0> and a __syncwarp)
__device__ __forceinline__ void fetch_tab(const Q8Params &p, const Unit &x, int *tab, int lane) {
  const int nent = tab_entries(p, x), first = x.tok0 >> p.block_shift;
  const int32_t *src = p.block_table + x.b * p.bt_stride + first;
#pragma unroll 1
  for (int e = lane; e < nent; e += 32) {
    if (first + e < p.max_blocks_per_seq)
      cp_async4(tab + e, src + e);
    else
      tab[e] = kPastWidth;
  }
}

__device__ __forceinline__ void load_scales(const Q8Params &p, const Unit &x, const int *tab,
                                            int (&kb)[kTabBatch], int (&vb)[kTabBatch], int lane) {
  const int nent = tab_entries(p, x);
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i) {
    const int64_t blk = lane + 32 * i < nent ? tab[lane + 32 * i] : -1;
    kb[i] = vb[i] = 127;
    if (blk >= 0 && blk < p.num_blocks) {  // (kPastWidth is negative)
      kb[i] = ldg_here(p.k_sc + blk * p.ksc_sb + x.kvh * p.ksc_sh);
      vb[i] = ldg_here(p.v_sc + blk * p.vsc_sb + x.kvh * p.vsc_sh);
    }
  }
}

__device__ __forceinline__ void put_scales(const Q8Params &p, const Unit &x, const int (&kb)[kTabBatch],
                                           const int (&vb)[kTabBatch], uint16_t *sctab, int lane) {
  const int nent = tab_entries(p, x);
#pragma unroll
  for (int i = 0; i < kTabBatch; ++i) {
    const int e = lane + 32 * i;
    if (e < nent)
      sctab[e] = static_cast<uint16_t>(checked_scale(kb[i], p.err) | (checked_scale(vb[i], p.err) << 8));
  }
}

// Offset of 16-byte chunk c of row r in a K-major operand of D-byte rows under
// the tile's swizzle.
template <int D>
__device__ __forceinline__ int swz16(int r, int c) {
  return r * D + ((D == 128 ? (c ^ (r & 7)) : (c ^ ((r >> 1) & 3))) << 4);
}

// The power of two that a query row is multiplied by, and its inverse, from the
// bits of the row's largest magnitude (ordered like the values, NaN and inf on
// top): that magnitude goes to [128, 256), exponent field + k = 127 + 7, with k
// held to [-60, 60] so that c 2^-k 2^ek stays a normal number (rows below 2^-53
// keep fewer bits, values past 2^68 saturate).  A row with an infinity or NaN
// is multiplied by 0: those elements become NaN, the rest zero.
struct QScale {
  float f, back;
};
__device__ __forceinline__ QScale q_scale(uint32_t top) {
  const bool finite = top < 0x7F80u;
  const int k = !finite || top == 0 ? 0 : max(-60, min(60, 134 - max(static_cast<int>(top >> 7), 1)));
  return QScale{finite ? __int_as_float((127 + k) << 23) : 0.f, __int_as_float((127 - k) << 23)};
}

// The query rows of unit x as q_hi and q_lo (the B operands of S^T) and their
// factors c 2^-k.  D / 8 lanes share a row, eight elements each; a pass of the
// warp takes 256 / D rows.  Rows past x.rows keep whatever the buffer holds:
// their columns of S^T are never used.
template <int D>
__device__ __forceinline__ const uint4 *q_row(const Q8Params &p, const Unit &x, int c) {
  const int r = x.row0 + c;
  const int i = r / p.G, g = r - i * p.G;
  return reinterpret_cast<const uint4 *>(p.q + q_tok_off(p, x, i) +
                                         static_cast<int64_t>(x.kvh * p.G + g) * p.q_sh);
}

template <int D, int N>
__device__ __forceinline__ void put_q_pass(const Q8Params &p, uint4 v, int c, uint8_t *qdst,
                                           float *rowf, int lane) {
  constexpr int kLanes = D / 8;
  const int ch = lane % kLanes;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;  // largest magnitude as bits: ordered like the values, NaN and inf on top
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const QScale qs = q_scale(top);
  const float f = qs.f;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const Split2 s = split_q(__fmul_rn(__uint_as_float(w[e] << 16), f),
                             __fmul_rn(__uint_as_float(w[e] & 0xFFFF0000u), f));
    hi[e] = s.hi;
    lo[e] = s.lo;
  }
  *reinterpret_cast<uint2 *>(qdst + swz16<D>(c, ch >> 1) + (ch & 1) * 8) =
      make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
  *reinterpret_cast<uint2 *>(qdst + swz16<D>(N + c, ch >> 1) + (ch & 1) * 8) =
      make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  if (ch == 0) rowf[c] = __fmul_rn(p.cscale, qs.back);
}

// The units of this CTA, in shared memory, where they were worked out once (the
// divisions of unit_make in every role would be most of the kernel's code).
// The host's grid leaves a CTA at most kSchedMaxMine of them.
struct Sched8 {
  const Unit *units;
  int count;
};

// First unit with tiles at or after `from`, or -1.
__device__ __forceinline__ int next_unit8(const Sched8 &sc, int from, Unit &out) {
  for (int k = from; k < sc.count; ++k) {
    out = sc.units[k];
    if (out.n_tiles > 0) return k;
  }
  return -1;
}

// The preparing warp: for every unit with tiles, in order, its table and scale
// bytes (slot unit % kUS) and its query rows (buffer unit % kQB).
template <class C>
__device__ __forceinline__ void prepare_q8(const Q8Params &p, uint8_t *smem, typename C::Small *sm,
                                           int lane, volatile int *abort_any, const Sched8 &sc) {
  constexpr int D = C::kD, N = C::kN, QB = C::kQB, US = C::kUS;
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes per query row, rows per pass
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    bool ok = true;
    if (lane == 0) ok = mbar_wait_call(bar, parity, abort_any, p.wait_ns);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
  };
  Unit cur, nxt;
  int k = next_unit8(sc, 0, cur);
  if (k >= 0) fetch_tab(p, cur, sm->tab[0], lane);
  cp_async_commit();
  int kb[kTabBatch], vb[kTabBatch];
  for (int ui = 0; k >= 0; ++ui) {
    const int nk = next_unit8(sc, k + 1, nxt);
    // this unit's query rows, and the next unit's table
#pragma unroll 1
    for (int c = lane / kLanes; c < cur.rows; c += kRows)
      cp_async16(sm->raw_q + c * D * 2 + (lane % kLanes) * 16, q_row<D>(p, cur, c) + lane % kLanes, 16);
    cp_async_commit();
    if (nk >= 0) {
      const int n = ui + 1;
      if (!wait(&sm->tab_free[n % US], ((n / US) & 1) ^ 1)) break;
      fetch_tab(p, nxt, sm->tab[n % US], lane);
    }
    cp_async_commit();
    cp_async_wait<2>();  // this unit's table
    __syncwarp();
    load_scales(p, cur, sm->tab[ui % US], kb, vb, lane);
    put_scales(p, cur, kb, vb, sm->sctab[ui % US], lane);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->tab_full[ui % US]);
    // Q goes into the buffer of the unit two before this one, once that unit's
    // last QK^T and its epilogue (staged there) are done and the softmax warps
    // have seen it
    if (!wait(&sm->q_empty[ui % QB], ((ui / QB) & 1) ^ 1)) break;
    cp_async_wait<1>();
    __syncwarp();
    uint8_t *dst = smem + C::kOffQ + (ui % QB) * C::kQBytes;
#pragma unroll 1
    for (int c0 = 0; c0 < cur.rows; c0 += kRows) {
      const int c = c0 + lane / kLanes;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (c < cur.rows)
        v = *reinterpret_cast<const uint4 *>(sm->raw_q + c * D * 2 + (lane % kLanes) * 16);
      put_q_pass<D, N>(p, v, c, dst, sm->rowf[ui % QB], lane);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->q_full[ui % QB]);
    cur = nxt;
    k = nk;
  }
  cp_async_wait<0>();
}

// One loading warp: K (with the tiles' scale bytes) or V of the tiles that go
// to its stages -- even or odd ones, or (kParts = 1) all: a stage has one warp, which then waits for
// every use of it in turn (a parity wait cannot tell a use from the one two
// before it).  Eight lanes (boxes) of a tile at once.  The bounded waits and
// the exit are those of attn_split.cuh's produce().
template <class C, int NS, int kParts>
__device__ __forceinline__ void load_q8(const Q8Params &p, const CUtensorMap *map, uint8_t *smem,
                                        typename C::Small *sm, uint64_t *full, uint64_t *empty,
                                        uint32_t dst_off, bool is_k, int part, int lane,
                                        volatile int *abort_any, const Sched8 &sc) {
  constexpr int D = C::kD, US = C::kUS;
  const int bmask = (1 << p.block_shift) - 1;
  if (lane == 0) tma_prefetch_desc(map);
  const uint32_t box_bytes = static_cast<uint32_t>(p.box_slots * D);
  int gi = 0;
  bool failed = false;
  Unit x;
  for (int k = next_unit8(sc, 0, x), ui = 0; k >= 0 && !failed;
       k = next_unit8(sc, k + 1, x), ++ui) {
    bool okt = true;
    if (lane == 0) okt = mbar_wait_call(&sm->tab_full[ui % US], (ui / US) & 1, abort_any, p.wait_ns);
    if (!__shfl_sync(0xffffffffu, okt ? 1 : 0, 0)) break;
    const int *tab = sm->tab[ui % US];
    const uint16_t *sct = sm->sctab[ui % US];
    for (int j = 0; j < x.n_tiles; ++j, ++gi) {
      const int st = gi % NS;
      if (kParts == 2 && (st & 1) != part) continue;
      bool okw = true;
      if (lane == 0) okw = mbar_wait_call(&empty[st], ((gi / NS) & 1) ^ 1, abort_any, p.wait_ns);
      if (!__shfl_sync(0xffffffffu, okw ? 1 : 0, 0)) {
        failed = true;
        break;
      }
      const int tok0 = x.tok0 + j * kTileTokens;
      const int nbox = (min(kTileTokens, x.lim_max - tok0) + p.box_slots - 1) >> p.box_shift;
      const int tok = tok0 + (lane << p.box_shift);
      int blk = 0, errs = 0;
      bool load = false;
      if (lane < nbox) {
        const int e = (tok - x.tok0) >> p.block_shift;
        blk = tab[e];
        if (blk == kPastWidth)
          errs = kErrTableWidth;
        else if (blk < 0 || static_cast<int64_t>(blk) >= p.num_blocks)
          errs = kErrBadBlock;
        else
          load = true;
        if (is_k) sm->sc[gi % C::kSC][lane] = sct[e];
      }
      const uint32_t loads = __ballot_sync(0xffffffffu, load);
      __syncwarp();  // (the scale bytes, before the arrival)
      if (lane == 0) {
        if (is_k) mbar_arrive(&sm->sc_full[gi % C::kSC]);
        mbar_arrive_expect_tx(&full[st], __popc(loads) * box_bytes);
      }
      __syncwarp();
      if (load) {
        const int slot = tok & bmask;
        tma_load_4d(smem + dst_off + st * C::kKVBytes + lane * box_bytes, map, &full[st], 0,
                    p.map_head_first ? x.kvh : slot, p.map_head_first ? slot : x.kvh, blk);
      }
      if (errs && p.err) atomicOr(p.err, errs);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->tab_free[ui % US]);
  }
  if (lane == 0) {
    // every copy this warp issued lands before the CTA exits (bounded): the
    // last tile of each of its stages
    volatile int no_abort = 0;
    for (int g = max(gi - NS, 0); g < gi; ++g)
      if (kParts == 1 || (g % NS & 1) == part) mbar_wait_call(&full[g % NS], (g / NS) & 1, &no_abort);
  }
}

template <int D, int N, int NSK, int NSV>
__global__ void __launch_bounds__(32 * Q8Cfg<D, N, NSK, NSV>::kWarps, 1)
    attn_split_q8_kernel(const __grid_constant__ Q8Params p,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v) {
  using C = Q8Cfg<D, N, NSK, NSV>;
  constexpr int QB = C::kQB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto *sm = reinterpret_cast<typename C::Small *>(smem + C::kOffSmall);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int *abort_any = &sm->abort_any;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NSK; ++i) {
      mbar_init(&sm->full_k[i], 1);
      mbar_init(&sm->empty_k[i], 1);
    }
    for (int i = 0; i < NSV; ++i) {
      mbar_init(&sm->full_v[i], 1);
      mbar_init(&sm->empty_v[i], 1);
    }
    for (int i = 0; i < C::kSC; ++i) mbar_init(&sm->sc_full[i], 1);
    for (int i = 0; i < C::kUS; ++i) {
      mbar_init(&sm->tab_full[i], 1);
      mbar_init(&sm->tab_free[i], C::kLoaders);
    }
    for (int i = 0; i < C::kSB; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->s_free[i], 4);   // one arrival per warp of a softmax warpgroup
    }
    for (int i = 0; i < C::kNP; ++i) {
      mbar_init(&sm->p_full[i], 4);   // one arrival per warp of a softmax warpgroup
      mbar_init(&sm->o_full[i], 1);
      mbar_init(&sm->stat_free[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->m_full[i], 4);   // one arrival per warp of a softmax warpgroup
      mbar_init(&sm->unit_done[i], 1);
      mbar_init(&sm->o_free[i], 4);   // one arrival per correction warp
      mbar_init(&sm->q_full[i], 1);
      // the unit's last QK^T, its epilogue, and every softmax warp
      mbar_init(&sm->q_empty[i], 2 + 4 * C::kNW);
      mbar_init(&sm->drain[i], 1);
    }
    sm->abort_any = 0;
    fence_barrier_init();
  }
  if (warp == C::kQkW) tmem_alloc(&sm->tmem_base, C::kTmemCols);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // In a packed call the row-major kernel's CTAs take the SMs over as this
  // grid's leave them (every CTA of it is resident or has been by now).
  if (threadIdx.x == 0) launch_dependents();
  const uint32_t tmem = sm->tmem_base;
  const uint32_t sbase = smem_u32(smem);
  // the Q and P^T buffers are not in use yet: the schedule's scratch
  Sched8 sc;
  {
    Sched deal = strided_sched(p);
    if (p.sched) {
      build_schedule<N>(p, smem + C::kOffQ, C::kSchedScratch, sm->sched_hist,
                        sm->sched_list, sm->sched_meta, &sm->sched_count);
      if (sm->sched_count >= 0) deal = Sched{sm->sched_list, sm->sched_meta, sm->sched_count};
    }
    sc = Sched8{sm->units, min(deal.count, kSchedMaxMine)};
    for (int k = threadIdx.x; k < sc.count; k += blockDim.x) sm->units[k] = deal.get<N>(p, k);
    __syncthreads();
  }

  if (warp == C::kPrepW) {
    prepare_q8<C>(p, smem, sm, lane, abort_any, sc);
  } else if (warp >= C::kLoadW && warp < C::kQkW) {
    const int w = warp - C::kLoadW;
    if (w < 2)
      load_q8<C, NSK, 2>(p, &map_k, smem, sm, sm->full_k, sm->empty_k, C::kOffK, true, w, lane, abort_any, sc);
    else
      load_q8<C, NSV, 2>(p, &map_v, smem, sm, sm->full_v, sm->empty_v, C::kOffV, false, w - 2, lane,
                      abort_any, sc);
  } else if (warp == C::kQkW || warp == C::kPvW) {
    // ------------------------------------------------------------------
    // MMA issuers, one thread each: QK^T of every tile as soon as its K and a
    // S^T buffer are there, and P.V of every tile as soon as its P and V are.
    // One thread for both spent 1750 cycles on a tile (issue of 12 small MMAs
    // and 5 commits, and the waits between), more than the 1500 that the
    // tile's 32 KB take from memory.
    // ------------------------------------------------------------------
    if (lane == 0) {
      const bool is_qk = warp == C::kQkW;
      // A = K tile, B = [q_hi | q_lo] (K-major); A = V^T, B = P^T (MN-major)
      constexpr uint32_t kQk = idesc_f8(128, C::kQCols, kFmtE4M3, kFmtE4M3, 0, 0);
      constexpr uint32_t kPv = idesc_f8(128, C::kPCols, kFmtE4M3, kFmtE5M2, 1, 1);
      int gi = 0, pi = 0, ui = 0;
      bool failed = false;
      for (int k = 0; k < sc.count && !failed; ++k) {
        const Unit x = sc.units[k];
        if (x.n_tiles == 0) continue;
        if (is_qk) {
          const int qb = ui % QB;
          if (!mbar_wait_call(&sm->q_full[qb], (ui / QB) & 1, abort_any, p.wait_ns)) {
            failed = true;
            break;
          }
          const uint64_t bh = smem_desc(sbase + C::kOffQ + qb * C::kQBytes, 16, C::kAtom, C::kLayout);
          for (int j = 0; j < x.n_tiles; ++j, ++gi) {
            const int st = gi % NSK, sb = gi % C::kSB;
            if (!mbar_wait_call(&sm->full_k[st], (gi / NSK) & 1, abort_any, p.wait_ns) ||
                !mbar_wait_call(&sm->s_free[sb], ((gi / C::kSB) & 1) ^ 1, abort_any, p.wait_ns)) {
              failed = true;
              break;
            }
            tc_fence_after_sync();
            const uint64_t a = smem_desc(sbase + C::kOffK + st * C::kKVBytes, 16, C::kAtom, C::kLayout);
            const uint32_t d = tmem + sb * C::kQCols;
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) umma_f8(d, a + kk * 2, bh + kk * 2, kQk, kk > 0 ? 1u : 0u);
            umma_commit(&sm->s_full[sb]);
            umma_commit(&sm->empty_k[st]);
            if (j == x.n_tiles - 1) umma_commit(&sm->q_empty[qb]);
          }
        } else {
          const int ob = ui & 1;
          const uint32_t d = tmem + C::kColO + ob * C::kPCols;
          if (!mbar_wait_call(&sm->o_free[ob], ((ui >> 1) & 1) ^ 1, abort_any, p.wait_ns)) {
            failed = true;
            break;
          }
          for (int j = 0; j < x.n_tiles; j += 2, ++pi) {
            const int bb = pi % C::kNP, nh = min(2, x.n_tiles - j);
            if (!mbar_wait_call(&sm->p_full[bb], (pi / C::kNP) & 1, abort_any, p.wait_ns)) {
              failed = true;
              break;
            }
            for (int h = 0; h < nh && !failed; ++h, ++gi) {
              const int st = gi % NSV;
              if (!mbar_wait_call(&sm->full_v[st], (gi / NSV) & 1, abort_any, p.wait_ns)) {
                failed = true;
                break;
              }
              tc_fence_after_sync();
              // V^T: MN-major, 32 tokens (four 8-token atoms) per step.  D = 64:
              // both M halves read the same 64 columns; lanes 64..127 are unused.
              const uint64_t a = smem_desc(sbase + C::kOffV + st * C::kKVBytes, 0, C::kAtom, C::kLayout);
              // P^T: MN-major, no swizzle; 16-column groups 128 B apart, 8-token
              // groups kPKGroup apart
              const uint64_t b = smem_desc(sbase + C::kOffP + bb * C::kPBytes + h * C::kPTile,
                                           C::kPKGroup, 128, kLayoutInterleave);
#pragma unroll
              for (int kk = 0; kk < kTileTokens / 32; ++kk)
                umma_f8(d, a + kk * (4 * C::kAtom >> 4), b + kk * (4 * C::kPKGroup >> 4), kPv,
                        (j == 0 && h == 0 && kk == 0) ? 0u : 1u);
              umma_commit(&sm->empty_v[st]);
            }
            umma_commit(&sm->o_full[bb]);
            if (j + 2 >= x.n_tiles) umma_commit(&sm->unit_done[ob]);
          }
        }
        ++ui;
      }
      // every MMA this thread issued completes before TMEM is released
      (void)failed;
      uint64_t *drain = &sm->drain[is_qk ? 0 : 1];
      umma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait_call(drain, 0, &no_abort);
    }
  } else if (warp < C::kCorr0) {
    // ------------------------------------------------------------------
    // Softmax warpgroups: warpgroup wg takes the pairs of tiles with pi % kNW
    // == wg; thread t <-> TMEM lane t <-> token t of either tile.
    // ------------------------------------------------------------------
    const int wg = warp >> 2, wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t bar_id = 1 + wg;
    const float NEG_INF = neg_inf();
    int gbase = 0, pbase = 0, uo = 0;  // uo: ordinal of the unit among this CTA's units with work
    bool stop = false;
    for (int k = 0; k < sc.count && !stop; ++k) {
      const Unit x = sc.units[k];
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
      // the unit's Q and row factors are staged.  (A warpgroup without a pair in
      // the unit waits too, and the unit's end does not wait for it: what keeps
      // the phase from moving on past it is its own arrival at q_empty below.)
      const bool okq = mbar_wait_call(&sm->q_full[uo % QB], (uo / QB) & 1, abort_any, p.wait_ns);
      const float *rowf = sm->rowf[uo % QB];
      if (wg_bar_or(bar_id, !okq)) {
        stop = true;
        break;
      }
      for (int j = 0; j < x.n_tiles; j += 2) {
        const int pi = pbase + (j >> 1);
        if (pi % C::kNW != wg) continue;
        const int g0 = gbase + j, bb = pi % C::kNP;
        const int use = pi / C::kNP;  // of the P^T buffer and the statistics beside it
        const bool two = j + 1 < x.n_tiles;
        bool ok = true;
        constexpr int kLd = 2 * N;  // S_hi and S_lo
        float sv[2][kLd];
        float ks[2], ev[2], vs[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 0 || two) {
            const int g = g0 + h, sb = g % C::kSB, sl = g % C::kSC;
            ok = mbar_wait_call(&sm->sc_full[sl], (g / C::kSC) & 1, abort_any, p.wait_ns) && ok;
            ok = mbar_wait_call(&sm->s_full[sb], (g / C::kSB) & 1, abort_any, p.wait_ns) && ok;
            tc_fence_after_sync();
            tmem_ld_cols<kLd>(tmem + lane_off + sb * C::kQCols, sv[h]);
          }
        }
        const int tok0 = x.tok0 + j * kTileTokens + t;  // token of the first tile; the second's is 128 on
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int sl = (g0 + h) % C::kSC;
          const int both = tok0 + h * kTileTokens < x.lim_max ? sm->sc[sl][t >> p.box_shift] : 127 | (127 << 8);
          ks[h] = scale_of(both & 255);
          ev[h] = static_cast<float>((both >> 8) - 127);
          vs[h] = scale_of(both >> 8);
        }
        tmem_ld_cols_wait<kLd>(sv[0]);
        if (two) tmem_ld_cols_wait<kLd>(sv[1]);
        // the S^T buffers are read
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm->s_free[g0 % C::kSB]);
          if (two) mbar_arrive(&sm->s_free[(g0 + 1) % C::kSB]);
        }
        if (x.tok0 + (j + 2) * kTileTokens > x.lim_max && j + 2 >= x.n_tiles) {
          // The unit's last tile: keys past the loaded range hold stale bytes;
          // once V has landed, zero those V rows so that 0 * V stays 0 in P.V.
          const int h = two ? 1 : 0, st = (g0 + h) % NSV;
          ok = mbar_wait_call(&sm->full_v[st], ((g0 + h) / NSV) & 1, abort_any, p.wait_ns) && ok;
          if (ok && tok0 + h * kTileTokens >= x.lim_max) {
            uint4 *vrow = reinterpret_cast<uint4 *>(smem + C::kOffV + st * C::kKVBytes + t * D);
#pragma unroll
            for (int k16 = 0; k16 < D / 16; ++k16) vrow[k16] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        float(*wmax)[N] = sm->wmax[wg][(pi / C::kNW) & 1];
#pragma unroll
        for (int q4 = 0; q4 < N / 4; ++q4) {
          const int4 lim = *reinterpret_cast<const int4 *>(&sm->lim[wg][4 * q4]);
          const float4 rf = *reinterpret_cast<const float4 *>(&rowf[4 * q4]);
          const int lims[4] = {lim.x, lim.y, lim.z, lim.w};
          const float rfs[4] = {rf.x, rf.y, rf.z, rf.w};
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 4 * q4 + e;
            v[e] = NEG_INF;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // (masked, a missing second tile, and rows past x.rows, whose
              // limit is 0: the score itself is -inf from here on)
              const bool seen = (h == 0 || two) && tok0 + h * kTileTokens < lims[e];
              sv[h][c] = seen ? join_q(sv[h][c], sv[h][N + c]) : NEG_INF;
              if (seen) v[e] = fmaxf(v[e], __fmaf_rn(sv[h][c], __fmul_rn(rfs[e], ks[h]), ev[h]));
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = warp_max(v[e]);
          if (lane == 0)
            *reinterpret_cast<float4 *>(&wmax[wq][4 * q4]) = make_float4(v[0], v[1], v[2], v[3]);
        }
        // P^T[bb] is free once P.V of pair pi - kNP is done, the row statistics
        // once the correction of that pair has read them
        ok = mbar_wait_call(&sm->o_full[bb], (use & 1) ^ 1, abort_any, p.wait_ns) && ok;
        ok = mbar_wait_call(&sm->stat_free[bb], (use & 1) ^ 1, abort_any, p.wait_ns) && ok;
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
        // the running references: the previous pair's, this pair's.  Every
        // warp works them out for itself (lane = row), so that the chain from
        // pair to pair has no barrier in it; warp 0 publishes them.
        if (pi > 0)
          ok = mbar_wait_call(&sm->m_full[(pi - 1) & 1], ((pi - 1) >> 1) & 1, abort_any, p.wait_ns) && ok;
        bool moved = false;
        float root = 1.f;
        if (lane < N) {
          const int c = lane;
          float m_new = NEG_INF, a = 1.f;
          if (c < x.rows) {
            const float tmax = fmaxf(fmaxf(wmax[0][c], wmax[1][c]), fmaxf(wmax[2][c], wmax[3][c]));
            const float m_prev = j > 0 ? sm->mrun[(pi - 1) & 1][c] : NEG_INF;
            m_new = (tmax > __fadd_rn(m_prev, kRefTop)) ? __fsub_rn(tmax, kRefDrop) : m_prev;
            if (m_prev != NEG_INF && m_new != m_prev) {
              const float d = __fsub_rn(m_prev, m_new);
              a = ex2(d);
              root = ex2(__fmul_rn(0.5f, d));
              moved = true;
            }
          }
          sm->mw[wg][wq][c] = m_new;
          if (wq == 0) {
            sm->mrun[pi & 1][c] = m_new;
            sm->mnew[bb][c] = m_new;
            sm->scl[bb][c] = root;
          }
          sm->aw[wg][wq][c] = a;
        }
        const bool resc = __any_sync(0xffffffffu, moved);
        __syncwarp();  // (mw / aw, for the warp)
        if (lane == 0) mbar_arrive(&sm->m_full[pi & 1]);
        if (resc) {
          // O^T holds the unit's earlier pairs once P.V of pair pi - 1 is done
          // (o_full of its buffer: the phase before is pair pi - 1 - kNP's, done
          // since that of pair pi - kNP was awaited above, and the one after
          // needs this pair)
          ok = mbar_wait_call(&sm->o_full[(pi - 1) % C::kNP], ((pi - 1) / C::kNP) & 1, abort_any, p.wait_ns) && ok;
          if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after_sync();
#pragma unroll 1
            for (int c0 = 0; c0 < C::kPCols; c0 += 16) {
              float o[16];
              tmem_ld16(ocol + c0, o);
              tmem_ld_wait_for(o);
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)  // (column c: row c % N; padding columns hold zeros)
                w[e] = __float_as_uint(__fmul_rn(o[e], sm->aw[wg][wq][(c0 + e) % N]));
              tmem_st16(ocol + c0, w);
            }
            tmem_st_wait();
          }
        }
        // P^T row t of either tile: bytes [hi | mid | lo] of the rows
        uint8_t *prow = smem + C::kOffP + bb * C::kPBytes + (t >> 3) * C::kPKGroup + (t & 7) * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[C::kPCols / 4];
#pragma unroll
          for (int i = 3 * N / 4; i < C::kPCols / 4; ++i) w[i] = 0u;
#pragma unroll
          for (int q4 = 0; q4 < N / 4; ++q4) {
            const float4 rf = *reinterpret_cast<const float4 *>(&rowf[4 * q4]);
            const float4 mm = *reinterpret_cast<const float4 *>(&sm->mw[wg][wq][4 * q4]);
            const float rfs[4] = {rf.x, rf.y, rf.z, rf.w}, ms[4] = {mm.x, mm.y, mm.z, mm.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float &s = sv[h][4 * q4 + i];
              s = (s == NEG_INF) ? 0.f : ex2(__fmaf_rn(s, __fmul_rn(rfs[i], ks[h]), -ms[i]));
            }
            const SplitP a = split_p(__fmul_rn(sv[h][4 * q4], vs[h]), __fmul_rn(sv[h][4 * q4 + 1], vs[h]));
            const SplitP b = split_p(__fmul_rn(sv[h][4 * q4 + 2], vs[h]), __fmul_rn(sv[h][4 * q4 + 3], vs[h]));
            w[q4] = a.hi | (b.hi << 16);
            w[N / 4 + q4] = a.mid | (b.mid << 16);
            w[N / 2 + q4] = a.lo | (b.lo << 16);
          }
#pragma unroll
          for (int i = 0; i < C::kPCols / 16; ++i)
            *reinterpret_cast<uint4 *>(prow + h * C::kPTile + i * 128) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        // the pair's row sums: e of both tiles, then a tree over the
        // lanes that halves the rows a lane carries twice (six shuffles for
        // four rows); lane 8 r holds row r
#pragma unroll
        for (int q4 = 0; q4 < N / 4; ++q4) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __fadd_rn(sv[1][4 * q4 + e], sv[0][4 * q4 + e]);
          const bool up = lane & 16, up2 = lane & 8;
          float a0 = up ? v[2] : v[0], a1 = up ? v[3] : v[1];
          a0 = __fadd_rn(a0, __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16));
          a1 = __fadd_rn(a1, __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16));
          float b = up2 ? a1 : a0;
          b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, up2 ? a0 : a1, 8));
#pragma unroll
          for (int off = 4; off >= 1; off >>= 1) b = __fadd_rn(b, __shfl_xor_sync(0xffffffffu, b, off));
          if ((lane & 7) == 0) sm->wsum[bb][wq][4 * q4 + (lane >> 3)] = b;
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->p_full[bb]);
      }
      if (stop) break;
      // this warp is through with the unit's Q buffer: its phase, its row factors
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_empty[uo % QB]);
      gbase += x.n_tiles;
      pbase += (x.n_tiles + 1) >> 1;
      ++uo;
    }
    (void)stop;
  } else if (warp < C::kPrepW) {
    // ------------------------------------------------------------------
    // Correction + epilogue warpgroup: thread r (< rows) owns row r's
    // running l; at the unit's end thread t <-> column d of O^T.
    // ------------------------------------------------------------------
    const int wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    constexpr uint32_t bar_id = 1 + C::kNW;
    const float NEG_INF = neg_inf();
    float acc[N];
    float m_run = NEG_INF, l_run = 0.f;
    int pbase = 0, cui = 0;
    bool bulk_out = false;   // thread 0 has bulk stores to complete before exit
    bool stop = false;
    for (int k = 0; k < sc.count && !stop; ++k) {
      const Unit x = sc.units[k];
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
      for (int j = 0; j < (x.n_tiles + 1) >> 1; ++j) {
        const int pi = pbase + j, bb = pi % C::kNP;
        const bool ok = mbar_wait_call(&sm->p_full[bb], (pi / C::kNP) & 1, abort_any, p.wait_ns);  // the pair's row statistics
        if (t < x.rows) {
          const float lt = __fadd_rn(__fadd_rn(sm->wsum[bb][0][t], sm->wsum[bb][1][t]),
                                     __fadd_rn(sm->wsum[bb][2][t], sm->wsum[bb][3][t]));
          const float root = sm->scl[bb][t];
          l_run = __fmaf_rn(__fmul_rn(l_run, root), root, lt);
          m_run = sm->mnew[bb][t];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->stat_free[bb]);  // the pair's statistics are read
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
      }
      if (stop) break;
      {
        const int ob = cui & 1;
        const bool ok = mbar_wait_call(&sm->unit_done[ob], (cui >> 1) & 1, abort_any, p.wait_ns);
        if (wg_bar_or(bar_id, !ok)) {
          stop = true;
          break;
        }
        tc_fence_after_sync();
        float o[3 * N];
        tmem_ld_cols<3 * N / 8 * 8>(tmem + lane_off + C::kColO + ob * C::kPCols, o);
        if constexpr (3 * N % 8 != 0) {
          float last[8];
          tmem_ld8(tmem + lane_off + C::kColO + ob * C::kPCols + 3 * N / 8 * 8, last);
          tmem_ld_wait_for8(last);
#pragma unroll
          for (int e = 3 * N / 8 * 8; e < 3 * N; ++e) o[e] = last[e % 8];
        }
        tmem_ld_cols_wait<3 * N / 8 * 8>(o);
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = join_p(o[c], o[N + c], o[2 * N + c]);
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
      pbase += (x.n_tiles + 1) >> 1;
    }
    // the partials are complete in global memory before the CTA leaves
    if (bulk_out) bulk_wait<0>();
    (void)stop;
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kQkW) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0 && sm->abort_any && p.err) atomicOr(p.err, kErrTimeout);
}

}  // namespace pkv
