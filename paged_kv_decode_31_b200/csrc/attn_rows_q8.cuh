// attn_rows_q8.cuh -- split-KV attention over an 8-bit paged cache with the
// query rows on the MMA's M axis, for calls with many rows per KV head (prefill
// chunks, packed prompts).
//
// Units, schedule, splits and merge are attn_split.cuh's, the cache and the
// scales attn_split_q8.cuh's.  128 rows r = i * G + g of one KV head against
// 128-token tiles:
//   S   = (q_hi + q_lo) K8^T   (kind::f8f6f4, M = 128 rows, N = 128 keys), the
//         query row times 2^k as two 8-bit operands of one scale
//         (split_q_one_scale), exact, into one fp32 accumulator;
//   w   = S (c 2^-k 2^ek) + ev per key (see attn_split_q8.cuh): the exponents
//         are those of a 16-key group at least, so a group's largest score
//         alone goes through the fused multiply-add to give its largest w;
//   m     rises to max(w) - kRowDrop when max(w) > m + kRefTop;
//   P   = fp16(2^(w - m)) <= 2^15 (off by at most 2^-11 relative, 2^-25
//         absolute, which is 2^-32 of a row's largest) over S in TMEM;
//   O  += P V16 (kind::f16), V16 the tile's e4m3 values as fp16, exactly;
//   l   = sum of 2^(w - m) 2^-ev in fp32, group sums first; a move of m scales
//         it in two steps (see attn_split_q8.cuh).
// Against the bf16 kernel, P is one operand where that takes two (an fp16 has
// the bits that a bf16 and its remainder are there for), so P.V is half the
// products, the softmax stores half the bytes and O is one accumulator, which
// leaves TMEM for a third S buffer.  V is widened because P in fp16 needs an
// fp16 partner; K is read in place.
//
// What bounds it: the length of a tile's chain, not a unit of the SM.  8 x 512
// queries at context 2048, Hq 16 / Hkv 4, D 128: 139.6 us, 430 TFLOP/s; 3300
// cycles a tile, of which the softmax's two passes take 2100, the exchange of
// the halves' maxima 120 and waits for S and the scale bytes 900, while the
// tensor pipe is at 23 %, issue at 49 % and the exponential pipe at 24 %: with
// one tile of rows per CTA nothing else runs beside its softmax.
// Code that stays small is what made it fast (start: 175 us; instruction-cache
// hits 71 % then, 84 % now): rolled softmax loops (-16), query rows converted a
// few at a time between V tiles and an epilogue of rolled 16-column steps without
// registers of its own for O, which also leaves the softmax 128 registers (-24).
// Measured and dropped: the two softmax warpgroups on alternate tiles (equal),
// 16 keys in flight ahead of those in use (+22), S kept in registers between the
// passes (+32), either pass unrolled (+2, +5), scales read inside the loops (+6).
//
// Roles (640 threads): warps 0-3 / 4-7 softmax (thread t = row t, keys [0, 64)
// and [64, 128) of every tile), 8-11 epilogue, 12-15 converters (V to fp16, and
// every unit's query rows to 8 bits), 16 K loader (+ scale bytes), 17 V loader,
// 18 MMA issuer + TMEM owner, 19 the units' tables and scales.
#pragma once

#include <type_traits>

#include "attn_rows.cuh"
#include "attn_split_q8.cuh"

namespace pkv {

constexpr int kR8Threads = 640;
// A row's largest P stays in [2^kRowDrop, 2^kRefTop] (see attn_split_q8.cuh):
// with [2^0, 2^8] the tokens 14 nats below it kept 4 bits of fp16 and fewer.
constexpr float kRowDrop = 7.f;
// P is flushed to zero below 2^-126, which must not take its P 2^-ev out of l:
// groups of keys with a scale below 2^kRowEvMin (blocks of zeros have 2^-63) go
// through the exponential with 2^kRowEvMin in its place, and P gets the rest
// afterwards.  What is flushed then is below 2^-102 of l's units, 2^-90 for a
// split's 4096 tokens, and l at least 2^(kRowDrop - 63).  (The form of
// attn_split_q8.cuh costs a product per element in the longest part of the
// chain: 146 us instead of 139.6 for 8 x 512 queries.)
constexpr float kRowEvMin = -24.f;
// Registers per thread: at launch, and each warpgroup's share of their sum.
constexpr int kR8LaunchRegs = 96, kR8SoftmaxRegs = 128, kR8EpiRegs = 88, kR8ConvRegs = 72, kR8AuxRegs = 64;
static_assert(2 * kR8SoftmaxRegs + kR8EpiRegs + kR8ConvRegs + kR8AuxRegs == 5 * kR8LaunchRegs,
              "warpgroup register shares must add up to the launch allocation");

template <int D>
struct R8Cfg {
  static constexpr int kD = D, kN = kRowsPerTile, kQB = 2;
  static constexpr int kEpi0 = 8, kConv0 = 12, kLoadK = 16, kLoadV = 17, kMma = 18, kPrep = 19;
  static constexpr int kLoaders = 2;
  static constexpr int NSK = D == 128 ? 3 : 6, NSV = D == 128 ? 2 : 4, NSH = D == 128 ? 2 : 4;
  static constexpr int kKVBytes = kTileTokens * D;      // an 8-bit tile
  static constexpr int kHBytes = kTileTokens * D * 2;   // an fp16 V tile: 64-wide halves
  static constexpr int kHalf = kTileTokens * 128;
  static constexpr uint32_t kLayout = D == 128 ? kLayoutSw128 : kLayoutSw64;
  static constexpr int kAtom = 8 * D;
  static constexpr int kQPiece = kRowsPerTile * D, kQBytes = 2 * kQPiece;
  static constexpr int kSB = 3;                          // S / P buffers
  static constexpr int kSC = 16, kUS = 2;
  static_assert(NSK + kSB <= kSC, "a slot of scale bytes is rewritten after its tile's softmax read it");
  static constexpr int kOffK = 0, kOffV = NSK * kKVBytes, kOffH = kOffV + NSV * kKVBytes,
                       kOffQ = kOffH + NSH * kHBytes, kOffSmall = kOffQ + kQB * kQBytes;
  static constexpr int kSchedScratch = kQB * kQBytes;    // bytes free at kernel start
  // also only at kernel start, in the fp16 tiles' place
  struct Start {
    int sched_list[kSchedMaxMine], sched_meta[kSchedMaxMine][3];
    int sched_hist[kSchedHist], sched_count;
  };
  static_assert(sizeof(Start) <= NSH * kHBytes, "start-up data");
  struct Small {
    uint64_t full_k[NSK], empty_k[NSK], full_v[NSV], empty_v[NSV], full_h[NSH], empty_h[NSH];
    uint64_t sc_full[kSC], tab_full[kUS], tab_free[kUS];
    uint64_t s_full[kSB], p_full[kSB], s_free[kSB];
    uint64_t ml_full[2], ml_free[2], unit_done, o_free;
    uint64_t q_full[2], q_empty[2], drain;
    uint32_t tmem_base;
    int abort_any;
    float xmax[2][2][kRowsPerTile];  // [tile parity][half][row]: the halves' maxima
    float xsum[2][kRowsPerTile];     // [tile parity][row]: the second half's sum
    float ml[2][2][kRowsPerTile];    // [unit parity][m, l][row]: the unit's final (m, l)
    float rowf[2][kRowsPerTile];     // [Q buffer][row]: c 2^-k
    Unit units[kSchedMaxMine];
    int tab[kUS][kSplitTokens / 16];
    uint16_t sctab[kUS][kSplitTokens / 16];
    uint16_t sc[kSC][8];
  };
  static constexpr int kSmemBytes = kOffSmall + static_cast<int>(sizeof(Small)) + 1024;
  static constexpr uint32_t kColO = kSB * 128;
};

// The end of row t of a 128-row tile: out and lse where the row has one split
// (the fold of one partial is the partial), else the partial.  16 columns of O
// at a time, in a loop that stays rolled: unrolled over the head it drove the
// softmax out of the instruction cache, and four to six tiles of every unit
// took half as long again.  out = O * (1 / l), not the merge's correctly
// rounded quotient: within 2^-23 of it before the rounding to bf16, and a
// tenth of the instructions while the softmax warps need every issue slot.
struct RowEnd {
  __nv_bfloat16 *out, *fin;  // final row (fin: the sequence's last row, or null)
  float *part;               // split partial (out is null)
  float inv;                 // 1 / l, 0 for a row that saw no key
};

__device__ __forceinline__ RowEnd row_end(const Q8Params &p, const Unit &x, int t, float m, float l, int D) {
  RowEnd r{};
  const int i = (x.row0 + t) / p.G, g = x.row0 + t - i * p.G, h = x.kvh * p.G + g;
  int lim = x.seqlen;
  if (p.causal) lim = min(lim, x.seqlen - x.nq + i + 1);
  if (lim > kSplitTokens) {
    const int64_t slot = ((x.q0 + i) * p.Hq + h) * static_cast<int64_t>(p.n_splits) + x.s;
    r.part = p.ws_acc + slot * D;
    *reinterpret_cast<float2 *>(p.ws_ml + slot * 2) = make_float2(m, l);
    return r;
  }
  if (x.s != 0) return r;
  r.inv = final_rcp(l);
  r.out = p.out + o_tok_off(p, x, i) + h * p.o_sh;
  const float ls = final_lse(m, l);
  p.lse[lse_index(p, x, i, h)] = ls;
  if (p.fin_out != nullptr && i == x.nq - 1) {
    r.fin = p.fin_out + x.b * p.fo_sb + h * p.fo_sh;
    p.fin_lse[static_cast<int64_t>(x.b) * p.Hq + h] = ls;
  }
  return r;
}

// 16 columns of O from column c on.
__device__ __forceinline__ void end_cols(const Q8Params &p, const RowEnd &r, int c, const float (&v)[16]) {
  if (r.part) {
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      *reinterpret_cast<float4 *>(r.part + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    return;
  }
  if (!r.out) return;
  __nv_bfloat162 h2[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    h2[e] = __floats2bfloat162_rn(__fmul_rn(v[2 * e], r.inv), __fmul_rn(v[2 * e + 1], r.inv));
  if (p.out_vec) {
    *reinterpret_cast<uint4 *>(r.out + c) = *reinterpret_cast<uint4 *>(h2);
    *reinterpret_cast<uint4 *>(r.out + c + 8) = *reinterpret_cast<uint4 *>(h2 + 4);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) r.out[c + e] = e & 1 ? h2[e >> 1].y : h2[e >> 1].x;
  }
  if (r.fin) {
#pragma unroll
    for (int e = 0; e < 16; ++e) r.fin[c + e] = e & 1 ? h2[e >> 1].y : h2[e >> 1].x;
  }
}

// Query rows of unit x as q_hi and q_lo, by the converter warpgroup, in place:
// the two halves of a row's bytes are copied to where its hi and its lo go
// (ask_q, asynchronous), then the D / 8 lanes that share a row read it and
// write both (put_q_rows: kQRows rows for 128 threads).  Rows past x.rows keep what the
// buffer holds: their S is not used.
template <int D>
constexpr int kQRows = 1024 / D;

template <int D>
__device__ __forceinline__ int raw_q_off(int r, int ch) {
  return (ch < D / 16 ? 0 : kRowsPerTile * D) + swz16<D>(r, ch % (D / 16));
}

// By NT threads: thread t takes chunk t % (D / 8) of rows t / (D / 8), ...
template <int D, int NT>
__device__ __forceinline__ void ask_q(const Q8Params &p, const Unit &x, int t, uint8_t *dst) {
  constexpr int kLanes = D / 8;
#pragma unroll 1
  for (int c = t / kLanes; c < x.rows; c += NT / kLanes)
    cp_async16(dst + raw_q_off<D>(c, t % kLanes), q_row<D>(p, x, c) + t % kLanes, 16);
  cp_async_commit();
}

template <int D, int NT>
__device__ __forceinline__ void put_q_rows(const Q8Params &p, int pass, int t, uint8_t *dst, float *rowf) {
  constexpr int kLanes = D / 8;
  const int ch = t % kLanes, c = pass * (NT / kLanes) + t / kLanes;
  const uint4 v = *reinterpret_cast<const uint4 *>(dst + raw_q_off<D>(c, ch));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
  for (int off = kLanes / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  const QScale qs = q_scale(top);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const Split2 a = split_q_one_scale(__fmul_rn(bf_lo(w[i]), qs.f), __fmul_rn(bf_hi(w[i]), qs.f));
    hi[i] = a.hi;
    lo[i] = a.lo;
  }
  __syncwarp();  // the row is read
  const int o = swz16<D>(c, ch >> 1) + (ch & 1) * 8;
  *reinterpret_cast<uint2 *>(dst + o) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
  *reinterpret_cast<uint2 *>(dst + kRowsPerTile * D + o) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
  if (ch == 0) rowf[c] = __fmul_rn(p.cscale, qs.back);
}

// An e4m3 V tile to fp16 (exact), 64-wide halves of 128-byte swizzled rows;
// tokens at or past `held` become zeros (their bytes are stale).
template <int D>
__device__ __forceinline__ void convert_v(const uint8_t *src, uint8_t *dst, int held, int t) {
  constexpr int kCh = D / 16;  // 16-byte chunks of a row
#pragma unroll 2
  for (int i = t; i < kTileTokens * kCh; i += 128) {
    const int tok = i / kCh, c = i % kCh;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (tok < held) v = *reinterpret_cast<const uint4 *>(src + swz16<D>(tok, c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 a = half2_of_e4m3x2(w[e] & 0xFFFFu), b = half2_of_e4m3x2(w[e] >> 16);
      o[2 * e] = *reinterpret_cast<const uint32_t *>(&a);
      o[2 * e + 1] = *reinterpret_cast<const uint32_t *>(&b);
    }
    uint8_t *row = dst + (c >> 2) * (kTileTokens * 128) + tok * 128;
    const int cc = (c & 3) * 2;
    *reinterpret_cast<uint4 *>(row + ((cc ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4 *>(row + (((cc + 1) ^ (tok & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <int D>
__global__ void __launch_bounds__(kR8Threads, 1)
    attn_rows_q8_kernel(const __grid_constant__ Q8Params p, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v) {
  using C = R8Cfg<D>;
  constexpr int NSK = C::NSK, NSV = C::NSV, NSH = C::NSH, SB = C::kSB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  auto *sm = reinterpret_cast<typename C::Small *>(smem + C::kOffSmall);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *abort_any = &sm->abort_any;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NSK; ++i) {
      mbar_init(&sm->full_k[i], 1);
      mbar_init(&sm->empty_k[i], 1);
    }
    for (int i = 0; i < NSV; ++i) {
      mbar_init(&sm->full_v[i], 1);
      mbar_init(&sm->empty_v[i], 4);  // one arrival per converter warp
    }
    for (int i = 0; i < NSH; ++i) {
      mbar_init(&sm->full_h[i], 4);
      mbar_init(&sm->empty_h[i], 1);
    }
    for (int i = 0; i < C::kSC; ++i) mbar_init(&sm->sc_full[i], 1);
    for (int i = 0; i < C::kUS; ++i) {
      mbar_init(&sm->tab_full[i], 1);
      mbar_init(&sm->tab_free[i], C::kLoaders);
    }
    for (int i = 0; i < SB; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->p_full[i], 8);  // one arrival per softmax warp
      mbar_init(&sm->s_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->q_full[i], 4);   // one arrival per converter warp
      mbar_init(&sm->q_empty[i], 9);  // the unit's last QK^T, and every softmax warp has its row factors
      mbar_init(&sm->ml_full[i], 4);
      mbar_init(&sm->ml_free[i], 4);
    }
    mbar_init(&sm->unit_done, 1);
    mbar_init(&sm->o_free, 4);
    mbar_init(&sm->drain, 1);
    sm->abort_any = 0;
    fence_barrier_init();
  }
  if (warp == C::kMma) tmem_alloc(&sm->tmem_base, 512);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm->tmem_base;
  const uint32_t sbase = smem_u32(smem);
  const float NEG_INF = neg_inf();
  Sched8 sc;
  {
    auto *start = reinterpret_cast<typename C::Start *>(smem + C::kOffH);
    Sched deal = strided_sched(p);
    if (p.sched) {
      build_schedule<kRowsPerTile>(p, smem + C::kOffQ, C::kSchedScratch, start->sched_hist, start->sched_list, start->sched_meta, &start->sched_count);
      if (start->sched_count >= 0) deal = Sched{start->sched_list, start->sched_meta, start->sched_count};
    }
    sc = Sched8{sm->units, min(deal.count, kSchedMaxMine)};
    for (int k = threadIdx.x; k < sc.count; k += kR8Threads) sm->units[k] = deal.get<kRowsPerTile>(p, k);
    __syncthreads();  // (also: the start-up data's place is free)
  }
  // The first unit's query rows, by the 16 warps that have nothing to do before
  // them (by the converters alone: 8 x 512 queries 137.4 us instead of 136.1)
  Unit first;
  const int k0 = next_unit8(sc, 0, first);
  if (warp < C::kLoadK && k0 >= 0) {
    constexpr int kStart = 32 * C::kLoadK;
    ask_q<D, kStart>(p, first, threadIdx.x, smem + C::kOffQ);
    cp_async_wait<0>();
    __syncwarp();
#pragma unroll 1
    for (int pass = 0; pass * (kStart / (D / 8)) < first.rows; ++pass)
      put_q_rows<D, kStart>(p, pass, threadIdx.x, smem + C::kOffQ, sm->rowf[0]);
    fence_proxy_async_smem();
    named_bar_or(4, kStart, false);
    if (warp >= C::kConv0 && lane == 0) mbar_arrive(&sm->q_full[0]);
  }

  if (warp >= C::kLoadK) {
    regs_dec<kR8AuxRegs>();
    if (warp == C::kLoadK) {
      load_q8<C, NSK, 1>(p, &map_k, smem, sm, sm->full_k, sm->empty_k, C::kOffK, true, 0, lane, abort_any, sc);
    } else if (warp == C::kLoadV) {
      load_q8<C, NSV, 1>(p, &map_v, smem, sm, sm->full_v, sm->empty_v, C::kOffV, false, 0, lane, abort_any, sc);
    } else if (warp == C::kPrep) {
      int kb[kTabBatch], vb[kTabBatch];
      Unit x;
      x = first;
      for (int k = k0, ui = 0; k >= 0;
           k = next_unit8(sc, k + 1, x), ++ui) {
        const int us = ui % C::kUS;
        bool ok = true;
        if (lane == 0) ok = mbar_wait(&sm->tab_free[us], ((ui / C::kUS) & 1) ^ 1, abort_any, p.wait_ns);
        if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) break;
        fetch_tab(p, x, sm->tab[us], lane);
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        load_scales(p, x, sm->tab[us], kb, vb, lane);
        put_scales(p, x, kb, vb, sm->sctab[us], lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->tab_full[us]);
      }
    } else if (lane == 0) {
      // ----------------------------------------------------------------
      // MMA issuer.  Per tile gi: S[gi % kSB] = Q K^T once the K stage has
      // landed and P.V of tile gi - kSB is done; then P.V of tile gi - (kSB -
      // 1), so that the softmax of two tiles can run meanwhile.
      // ----------------------------------------------------------------
      constexpr uint32_t kQkHi = idesc_f8(128, 128, kFmtE4M3, kFmtE4M3, 0, 0);  // A = q_hi, B = K
      constexpr uint32_t kQkLo = idesc_f8(128, 128, kFmtE5M2, kFmtE4M3, 0, 0);  // A = q_lo
      constexpr uint32_t kPv = idesc_f16(128, D, 0, 1);                         // A = P (TMEM), B = V (MN-major)
      struct Pend {
        int g, first, last, uo;
      };
      int gi = 0, ui = 0, npend = 0;
      Pend pend[2] = {{-1, 0, 0, 0}, {-1, 0, 0, 0}};
      bool failed = false;
      auto pv_step = [&](const Pend &pd) -> bool {
        const int g = pd.g, st = g % NSH, bb = g % SB;
        if (!mbar_wait(&sm->p_full[bb], (g / SB) & 1, abort_any, p.wait_ns)) return false;
        if (pd.first && !mbar_wait(&sm->o_free, (pd.uo & 1) ^ 1, abort_any, p.wait_ns)) return false;
        if (!mbar_wait(&sm->full_h[st], (g / NSH) & 1, abort_any, p.wait_ns)) return false;
        tc_fence_after_sync();
        const uint64_t b = smem_desc(sbase + C::kOffH + st * C::kHBytes, C::kHalf, 1024, kLayoutSw128);
#pragma unroll
        for (int kk = 0; kk < kTileTokens / 16; ++kk)
          // P of keys [16 kk, 16 kk + 16): TMEM columns 32 (kk / 2) + 8 (kk % 2) + [0, 8)
          umma_bf16_ts(tmem + C::kColO, tmem + bb * 128 + (kk >> 1) * 32 + (kk & 1) * 8, b + kk * (2048 >> 4), kPv,
                       (pd.first && kk == 0) ? 0u : 1u);
        umma_commit(&sm->empty_h[st]);
        umma_commit(&sm->s_free[bb]);
        if (pd.last) umma_commit(&sm->unit_done);
        return true;
      };
      for (int k = 0; k < sc.count && !failed; ++k) {
        const Unit x = sc.units[k];
        if (x.n_tiles == 0) continue;
        const int qb = ui & 1;
        if (!mbar_wait(&sm->q_full[qb], (ui >> 1) & 1, abort_any, p.wait_ns)) {
          failed = true;
          break;
        }
        const uint64_t qd = smem_desc(sbase + C::kOffQ + qb * C::kQBytes, 16, C::kAtom, C::kLayout);
        for (int j = 0; j < x.n_tiles; ++j, ++gi) {
          const int st = gi % NSK, bb = gi % SB;
          if (!mbar_wait(&sm->full_k[st], (gi / NSK) & 1, abort_any, p.wait_ns) ||
              !mbar_wait(&sm->s_free[bb], ((gi / SB) & 1) ^ 1, abort_any, p.wait_ns)) {
            failed = true;
            break;
          }
          tc_fence_after_sync();
          const uint64_t kd = smem_desc(sbase + C::kOffK + st * C::kKVBytes, 16, C::kAtom, C::kLayout);
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk) {
            umma_f8(tmem + bb * 128, qd + kk * 2, kd + kk * 2, kQkHi, kk > 0 ? 1u : 0u);
            umma_f8(tmem + bb * 128, qd + (C::kQPiece >> 4) + kk * 2, kd + kk * 2, kQkLo, 1u);
          }
          umma_commit(&sm->s_full[bb]);
          umma_commit(&sm->empty_k[st]);
          if (j == x.n_tiles - 1) umma_commit(&sm->q_empty[qb]);
          if (npend == SB - 1) {
            if (!pv_step(pend[0])) {
              failed = true;
              break;
            }
            pend[0] = pend[1];
            --npend;
          }
          pend[npend++] = Pend{gi, j == 0 ? 1 : 0, j == x.n_tiles - 1 ? 1 : 0, ui};
        }
        ++ui;
      }
      for (int i = 0; i < npend && !failed; ++i) failed = !pv_step(pend[i]);
      (void)failed;
      // every MMA this thread issued completes before TMEM is released
      umma_commit(&sm->drain);
      volatile int no_abort = 0;
      mbar_wait(&sm->drain, 0, &no_abort);
    }
  } else if (warp >= C::kConv0) {
    // ------------------------------------------------------------------
    // Converters: every V tile to fp16, and between a unit's first tiles the
    // next unit's query rows, a few passes each (in one go, a thread per row,
    // they held the V tiles up for 12000 cycles a unit).
    // ------------------------------------------------------------------
    regs_dec<kR8ConvRegs>();
    constexpr int kAtOnce = 2;  // passes per tile
    const int t = threadIdx.x & 127;
    Unit cur = first, nxt;
    if (k0 < 0) cur.n_tiles = 0;
    int k = k0 < 0 ? -1 : next_unit8(sc, k0 + 1, nxt), gi = 0;
    bool failed = false;
    for (int ord = 1; !failed; ++ord) {  // nxt: the CTA's ord-th unit with tiles, from 0
      uint8_t *qdst = smem + C::kOffQ + (ord & 1) * C::kQBytes;
      // passes over its rows; -1: they are not asked for yet
      const int passes = k >= 0 ? (nxt.rows + kAtOnce * kQRows<D> - 1) / (kAtOnce * kQRows<D>) * kAtOnce : 0;
      int pass = k >= 0 ? -1 : 0;
      for (int j = 0; j < cur.n_tiles || pass < passes; ++j) {
        bool ok = true;
        if (j < cur.n_tiles) {
          const int st = gi % NSV, sh = gi % NSH;
          ok = mbar_wait(&sm->full_v[st], (gi / NSV) & 1, abort_any, p.wait_ns) &&
               mbar_wait(&sm->empty_h[sh], ((gi / NSH) & 1) ^ 1, abort_any, p.wait_ns);
          failed = !__all_sync(0xffffffffu, ok);  // (a warp goes on, or gives up, as one)
          if (failed) break;
          convert_v<D>(smem + C::kOffV + st * C::kKVBytes, smem + C::kOffH + sh * C::kHBytes,
                       cur.lim_max - (cur.tok0 + j * kTileTokens), t);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm->full_h[sh]);
            mbar_arrive(&sm->empty_v[st]);
          }
          ++gi;
        }
        if (pass < 0) {
          ok = mbar_wait(&sm->q_empty[ord & 1], ((ord >> 1) & 1) ^ 1, abort_any, p.wait_ns);
          failed = !__all_sync(0xffffffffu, ok);
          if (failed) break;
          ask_q<D, 128>(p, nxt, t, qdst);
          pass = 0;
        } else if (pass < passes) {
          cp_async_wait<0>();
          __syncwarp();
#pragma unroll
          for (int e = 0; e < kAtOnce; ++e, ++pass) put_q_rows<D, 128>(p, pass, t, qdst, sm->rowf[ord & 1]);
          if (pass == passes) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm->q_full[ord & 1]);
          }
        }
      }
      if (k < 0) break;
      cur = nxt;
      k = next_unit8(sc, k + 1, nxt);
    }
    cp_async_wait<0>();
  } else if (warp < C::kEpi0) {
    // ------------------------------------------------------------------
    // Softmax warpgroups (see attn_rows.cuh for the exchange of the halves'
    // maxima and sums): thread t owns row t, warpgroup wg its keys [64 wg, 64
    // wg + 64).  O is rescaled half and half.
    // ------------------------------------------------------------------
    regs_inc<kR8SoftmaxRegs>();
    const int wg = warp >> 2, wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t ocol = tmem + lane_off + C::kColO + wg * (D / 2);
    constexpr uint32_t kXchgBar = 1, kDoneBar = 2;
    int gbase = 0, uo = 0;
    bool stop = false;
    for (int k = 0; k < sc.count && !stop; ++k) {
      const Unit x = sc.units[k];
      if (x.n_tiles == 0) continue;
      int nlim = 0;  // keys [0, nlim) are visible to row t
      if (t < x.rows) {
        const int i = (x.row0 + t) / p.G;
        int lim = x.seqlen;
        if (p.causal) lim = min(lim, x.seqlen - x.nq + i + 1);
        nlim = lim > 0 ? lim : 0;
      }
      bool okq = mbar_wait(&sm->q_full[uo & 1], (uo >> 1) & 1, abort_any, p.wait_ns);
      const float rf = t < x.rows ? sm->rowf[uo & 1][t] : 1.f;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->q_empty[uo & 1]);
      const bool live = 32 * wq < x.rows;  // (a warp without rows leaves its S and O as they are)
      float m_run = NEG_INF, l_run = 0.f;
      float root_prev = 1.f, half_prev = 0.f;
      for (int j = 0; j < x.n_tiles; ++j) {
        const int gi = gbase + j, bb = gi % SB, sl = gi % C::kSC;
        bool ok = mbar_wait(&sm->sc_full[sl], (gi / C::kSC) & 1, abort_any, p.wait_ns) && okq;
        ok = mbar_wait(&sm->s_full[bb], (gi / SB) & 1, abort_any, p.wait_ns) && ok;
        tc_fence_after_sync();
        const int tok0 = x.tok0 + j * kTileTokens;
        const int nvis = min(max(nlim - tok0, 0), kTileTokens);
        const uint32_t srow = tmem + lane_off + bb * 128;  // S of this tile, then its P
        // the scales of this half's four 16-key groups (keys past the loaded
        // range: any in range, their scores are masked)
        float f[4], ev[4], iv[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = 64 * wg + 16 * q;
          const int both = tok0 + key < x.lim_max ? sm->sc[sl][key >> p.box_shift] : 127 | (127 << 8);
          f[q] = __fmul_rn(rf, scale_of(both & 255));
          ev[q] = static_cast<float>((both >> 8) - 127);
          iv[q] = inv_scale_of(max(both >> 8, 127 + static_cast<int>(kRowEvMin)));
        }
        // pass 1: this half's largest w (the fused multiply-add rounds
        // monotonically, so a group's largest score gives its largest w).
        // The branch is taken per WARP (tcgen05.ld is .sync.aligned).
        __syncwarp();
        const bool full = __all_sync(0xffffffffu, nvis == kTileTokens);  // warp-uniform
        float hm = NEG_INF;
#pragma unroll 1
        for (int q = live ? 0 : 4; q < 4; q += 2) {
          float v0[16], v1[16];
          tmem_ld16(srow + 64 * wg + 16 * q, v0);
          tmem_ld16(srow + 64 * wg + 16 * q + 16, v1);
          tmem_ld_wait_for(v0);
          tmem_ld_wait_for(v1);
          if (!full) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              v0[e] = (64 * wg + 16 * q + e < nvis) ? v0[e] : NEG_INF;
              v1[e] = (64 * wg + 16 * q + 16 + e < nvis) ? v1[e] : NEG_INF;
            }
          }
          float r0 = v0[0], r1 = v1[0];
#pragma unroll
          for (int e = 1; e < 16; ++e) {
            r0 = fmaxf(r0, v0[e]);
            r1 = fmaxf(r1, v1[e]);
          }
          const float fa = q ? f[2] : f[0], fb = q ? f[3] : f[1], ea = q ? ev[2] : ev[0], eb = q ? ev[3] : ev[1];
          if (r0 != NEG_INF) hm = fmaxf(hm, __fmaf_rn(r0, fa, ea));
          if (r1 != NEG_INF) hm = fmaxf(hm, __fmaf_rn(r1, fb, eb));
        }
        sm->xmax[gi & 1][wg][t] = hm;
        if (named_bar_or(kXchgBar, 256, !ok)) {
          stop = true;
          break;
        }
        if (wg == 0 && j > 0)
          l_run = __fmaf_rn(__fmul_rn(l_run, root_prev), root_prev, __fadd_rn(half_prev, sm->xsum[(gi - 1) & 1][t]));
        const float mx = fmaxf(hm, sm->xmax[gi & 1][wg ^ 1][t]);
        const float m_prev = m_run;
        const float m_new = (mx > __fadd_rn(m_prev, kRefTop)) ? __fsub_rn(mx, kRowDrop) : m_prev;
        m_run = m_new;
        const float d = (m_prev == NEG_INF || m_new == m_prev) ? 0.f : __fsub_rn(m_prev, m_new);
        float root = 1.f;  // the factor of l, twice
        if (__any_sync(0xffffffffu, d != 0.f)) {
          root = d != 0.f ? ex2(__fmul_rn(0.5f, d)) : 1.f;
          const float a = d != 0.f ? ex2(d) : 1.f;
          // O holds the unit's tiles < gi once P.V(gi - 1) completes (s_free of
          // its buffer; see attn_rows.cuh on the parity)
          ok = mbar_wait(&sm->s_free[(gi - 1) % SB], ((gi - 1) / SB) & 1, abort_any, p.wait_ns) && ok;
          if (__all_sync(0xffffffffu, ok)) {
            tc_fence_after_sync();
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              float o[16];
              tmem_ld16(ocol + ch * 16, o);
              tmem_ld_wait_for(o);
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__fmul_rn(o[e], a));
              tmem_st16(ocol + ch * 16, w);
            }
          }
        }
        // pass 2: P over S, and this half's sum of P 2^-ev
        float half = 0.f;
        auto pass2 = [&](auto low) {
#pragma unroll 1
          for (int g2 = live ? 0 : 2; g2 < 2; ++g2) {  // 32 keys
            float v[2][16];
            tmem_ld16(srow + 64 * wg + 32 * g2, v[0]);
            tmem_ld16(srow + 64 * wg + 32 * g2 + 16, v[1]);
            tmem_ld_wait_for(v[0]);
            tmem_ld_wait_for(v[1]);
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int q = 2 * g2 + h;
              const float fq = g2 ? f[2 + h] : f[h], iq = g2 ? iv[2 + h] : iv[h], evq = g2 ? ev[2 + h] : ev[h];
              const float c = __fsub_rn(low ? fmaxf(evq, kRowEvMin) : evq, m_new);
#pragma unroll
              for (int e = 0; e < 16; ++e) v[h][e] = ex2(__fmaf_rn(v[h][e], fq, c));
              if (!full) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  v[h][e] = (64 * wg + 16 * q + e < nvis) ? v[h][e] : 0.f;
              }
              const float rest = low ? ex2(fminf(__fsub_rn(evq, kRowEvMin), 0.f)) : 1.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __half2 h2 = low ? __floats2half2_rn(__fmul_rn(v[h][2 * e], rest), __fmul_rn(v[h][2 * e + 1], rest))
                                       : __floats2half2_rn(v[h][2 * e], v[h][2 * e + 1]);
                w[8 * h + e] = *reinterpret_cast<const uint32_t *>(&h2);
              }
#pragma unroll
              for (int off = 8; off >= 1; off >>= 1)
#pragma unroll
                for (int e = 0; e < off; ++e) v[h][e] = __fadd_rn(v[h][e], v[h][e + off]);
              half = __fmaf_rn(v[h][0], iq, half);
            }
            tmem_st16(srow + 64 * wg + 32 * g2, w);
          }
        };
        if (fminf(fminf(ev[0], ev[1]), fminf(ev[2], ev[3])) < kRowEvMin)  // (warp-uniform)
          pass2(std::true_type{});
        else
          pass2(std::false_type{});
        if (wg == 1) sm->xsum[gi & 1][t] = half;
        const bool last = j == x.n_tiles - 1;
        if (last) {
          if (named_bar_or(kDoneBar, 256, !ok)) {
            stop = true;
            break;
          }
          if (wg == 0) {
            l_run = __fmaf_rn(__fmul_rn(l_run, root), root, __fadd_rn(half, sm->xsum[gi & 1][t]));
            // the slot of unit uo - 2 has been read by the epilogue
            ok = mbar_wait(&sm->ml_free[uo & 1], ((uo >> 1) & 1) ^ 1, abort_any, p.wait_ns) && ok;
            sm->ml[uo & 1][0][t] = m_run;
            sm->ml[uo & 1][1][t] = l_run;
          }
        } else {
          root_prev = root;
          half_prev = half;
        }
        __syncwarp();
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm->p_full[bb]);
          if (wg == 0 && last) mbar_arrive(&sm->ml_full[uo & 1]);
        }
      }
      gbase += x.n_tiles;
      ++uo;
    }
    (void)stop;
  } else {
    // ------------------------------------------------------------------
    // Epilogue warpgroup: thread t takes row t of each unit once its last P.V
    // is done, while the next unit's tiles already run.
    // ------------------------------------------------------------------
    regs_dec<kR8EpiRegs>();
    const int wq = warp & 3, t = threadIdx.x & 127;
    const uint32_t orow = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::kColO;
    constexpr uint32_t bar_id = 3;
    int uo = 0;
    for (int k = 0; k < sc.count; ++k) {
      const Unit x = sc.units[k];
      if (t == 0) check_sequence(p, x);
      const bool any = x.n_tiles > 0;  // (without a tile: out = 0, lse = -inf, by the unit of split 0)
      float m = NEG_INF, l = 0.f;
      if (any) {
        bool ok = mbar_wait(&sm->ml_full[uo & 1], (uo >> 1) & 1, abort_any, p.wait_ns);
        m = sm->ml[uo & 1][0][t];
        l = sm->ml[uo & 1][1][t];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->ml_free[uo & 1]);
        ok = mbar_wait(&sm->unit_done, uo & 1, abort_any, p.wait_ns) && ok;
        if (wg_bar_or(bar_id, !ok)) break;
        tc_fence_after_sync();
      }
      RowEnd r{};
      if (t < x.rows && (any || x.s == 0)) r = row_end(p, x, t, m, l, D);
#pragma unroll 1
      for (int c = 32 * wq < x.rows ? 0 : D; c < D; c += 16) {
        float v[16];
        __syncwarp();
        if (any) {
          tmem_ld16(orow + c, v);
          tmem_ld_wait_for(v);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.f;
        }
        end_cols(p, r, c, v);
      }
      if (any) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->o_free);
        ++uo;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == C::kMma) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sm->abort_any && p.err) atomicOr(p.err, kErrTimeout);
  // (a grid that overlaps the decode kernel's before it ends after it, so what
  // follows on the stream finds both complete)
  wait_for_grids_before();
}

}  // namespace pkv
